// Attention of the newest tokens of each request over its pages of the
// key-value cache.
//
// For a row at position p: o = Σ_t 2^(s_t − m) v_t / Σ_t 2^(s_t − m) over the
// tokens it sees, s_t = scale · log2(e) · q·k_t, in one pass over the tokens.
// m is a reference near the largest score so far: where a score exceeds it by
// more than 8, it moves up to the largest, from m to m', and sums and values
// so far are multiplied by 2^(m − m'); weights stay below 2⁸ and fp32 sums
// carry them as well as those below 1.
//
// Every byte of keys and values is used for a few rows only (query heads per
// key-value head × new tokens), so the pass is bound by reading the cache.
// The work is the list of all (request, key-value head, row tile, 64 tokens),
// in that order, cut into equal pieces, one for each CTA of a grid that is
// resident at once: requests of any lengths load every SM alike.  Items that
// several pieces share leave their sums in the workspace, and the CTA that
// finishes last joins them, sixteen at a time.  (SMs differ in how fast they
// read, ±12 % here; two further rounds of smaller pieces evened that out but
// cost more in starts and ends of pieces: 121 against 106 µs for 131071
// tokens.)
//
// Inside a CTA each group of R warps (16 query rows each) streams its own
// tokens through its own ring of cp.async copies, keys and values in turn, so
// that no barrier of the whole CTA stands in the loop; products run on
// m16n8k16 MMAs from registers, rows (at most 16·R) as their M, padded with
// zeros.  Every warp loads for itself: one warp that issued TMA copies for
// eight moved 3.5 TB/s, eight warps' cp.async 6.4.
//
// One request of 131071 tokens, 64 query and 8 key-value heads of 128: 100 µs
// (5.4 TB/s); 64 requests of up to 16384, 40 heads: 114 µs (5.6), in 8 bits
// 75 µs (4.4: bound by decoding, for 16 rows of which 5 exist); 96 requests that see 1024 tokens, 16 and 4
// heads of 256: 43 µs (3.4: half of it starts and ends of items).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "w4_attn_common.cuh"
#include "w4_attn_tc.h"
#include "w4_device.cuh"
#include "w4_kv.h"

namespace w4 {
namespace {

// (4, 2 or 1, for as many warps on an SM: 102, 110, 122 µs for one long request, 115, 119, 122 for 64 ragged ones,
// 84, 85, 89 in 8 bits, 45, 43, 64 for windows)
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 64;       // tokens of a unit of work
// Format 8's weights (times value scales) are at most 2⁸ of the reference and enter their products as fp16, below 65504
// and with 11 bits down to 2⁻¹⁴ only: they are taken 2⁷ times as large, and the outputs back at an item's end.
constexpr float kLift = 7.f, kLower = 0.0078125f;

// ------------------------------------------------------------- small pieces
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(~0u, v, 1));
    return fmaxf(v, __shfl_xor_sync(~0u, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(~0u, v, 1);
    return v + __shfl_xor_sync(~0u, v, 2);
}

// Two codes (biased by 128, in bytes `sel` of w) as fp16: 0x6400 | u is
// 1024 + u, exact, and so is the difference.
__device__ __forceinline__ uint32_t codes_f16(uint32_t w, uint32_t sel) {
    const uint32_t u = __byte_perm(w, 0x64646464u, sel);
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&u), bias);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// ------------------------------------------------------------------ kernel
// Shapes of the pass for head_dim ≤ D, R warps (16 rows each) per group.
template <int D, bool Q8, int R>
struct Shape {
    static constexpr int kGroups = kWarps / R;
    static constexpr int kElt = Q8 ? 1 : 2;
    static constexpr int kSub = D == 64 || (Q8 && D == 128) ? 2 : 1;  // 16-token blocks of a stage
    static constexpr int kTokens = 16 * kSub;
    static constexpr int kRow = D * kElt;            // bytes
    static constexpr int kChunks = kRow / 16;
    // An item's fixed cost (its first loads' latency, its sums' way out) in units of 64 tokens: about that of 96 KB of
    // keys and values.  64 ragged requests in 8 bits (16 KB a unit): 107, 93, 84, 86, 92 µs with 2, 3, 5, 8, 12;
    // in bf16 115, 116, 116, 117, 117; a window at head_dim 256 (64 KB): 48, 47, 50, 52, 56.
    static constexpr int kFixed = kRow >= 512 ? 2 : kRow == 256 ? 3 : kRow == 128 ? 6 : 10;
    static constexpr int kHalf = kTokens * kRow;     // a slot of the ring: a stage's keys or values
    // Three CTAs of 168 registers on an SM, where the outputs' D / 2 leave that; else two.  (Format 8 at D = 128, three
    // and two: 84 and 91 µs for 64 ragged requests.)
    static constexpr int kCtas = D == 256 ? 2 : 3;
    static constexpr int kBudget = (kCtas == 3 ? 72 : 108) * 1024;
    // Format 8 keeps the queries (as fp16, in the products' order) in shared memory: its decoding needs the registers.
    static constexpr int kQueries = Q8 ? R * (D / 16) * 512 : 0;
    static constexpr int kFit = (kBudget - kQueries) / (kGroups * (kHalf + (Q8 ? kTokens * 8 : 0)));
    static constexpr int kSlots = kFit > 12 ? 12 : Q8 ? kFit & ~1 : kFit;
    static constexpr int kAhead = (kSlots + 1) / 2;  // stages whose keys may be under way or in use
    static constexpr int kRing = kSlots * kHalf;
    // (key scale, log2 of value scale) of each token, for the stages on the way and the one in use
    static constexpr int kScaleSlots = kAhead + 1;
    static constexpr int kScales = Q8 ? kScaleSlots * kTokens * 8 : 0;
    static constexpr int kGroup = kRing + kScales;
    // Where the groups' sums meet: rows 8 columns apart in banks, and two numbers for each row.
    static constexpr int kMeetRow = D + 8, kMerge = kWarps * 16 * (kMeetRow + 2) * 4;
    static constexpr int kMain = kGroups * kGroup > kMerge ? kGroups * kGroup : kMerge, kSmem = kMain + kQueries;
    static_assert(kSlots >= 3 && (!Q8 || kSlots % 2 == 0), "a slot in use, two on the way; scales in time");
};

// Chunk c (of 16 bytes) of token row r lies at r · row + ((c ^ turn(r)) · 16):
// the loads of eight lanes that a shared-memory access serves at once fall in
// different banks.  turn(r) < 8 (4 for rows of 64 bytes) moves a chunk within
// 128 (64) bytes.
template <int ROW, bool Q8, bool KEY>
__device__ __forceinline__ int turn(int r) {
    return ROW == 64 ? (KEY ? 0 : (r >> 1) & 3) : Q8 && KEY ? ((r & 1) << 2) | ((r >> 1) & 3) : r & 7;
}

template <int R>
__device__ __forceinline__ void group_sync(int group) {
    if (R == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(R * 32) : "memory");
}

template <int D, bool Q8, int R>
__global__ void __launch_bounds__(kThreads, Shape<D, Q8, R>::kCtas) attn_split_kernel(const __grid_constant__ SplitArgs sp) {
    using S = Shape<D, Q8, R>;
    constexpr int NT = D / 8;   // output tiles of 8 columns
    constexpr int KS = D / 16;  // k-steps of 16
    constexpr int kRow = S::kRow, kFixed = S::kFixed;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ bool s_last, s_more;
    __shared__ Walk<kTile, 16 * R, S::kFixed> s_walk;
    __shared__ Item s_item[2];  // this item and the next: read again after the tokens, whose loop has no registers to spare
    const AttnArgs& a = sp.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int group = warp / R, rw = warp % R, G = sp.G;
    Walk<kTile, 16 * R, kFixed> walk;
    if (!walk.template find<kThreads>(sp)) return;
    bool more;
    {
        Item it;
        more = walk.next(sp, it);
        if (tid == 0) {
            s_walk = walk;
            s_item[0] = it;
        }
    }
    __syncthreads();

    const uint32_t ring = smem_addr(smem) + group * S::kGroup;
    float2* scales = reinterpret_cast<float2*>(smem + group * S::kGroup + S::kRing);
    uint4* queries = reinterpret_cast<uint4*>(smem + S::kMain);
    const int d_chunks = a.head_dim * S::kElt / 16;
    // The lane's places in a slot: of its 16 bytes of a copy's pass, and of what it reads.
    constexpr int kPerPass = 32 * R / S::kChunks;  // token rows of one pass of the group's lanes
    const int load_c = (rw * 32 + lane) % S::kChunks, load_r = (rw * 32 + lane) / S::kChunks;

    auto query_row = [&](const Item& n, int row) {
        const int j = sp.over_G(row);
        return a.q.data + (n.start + j) * a.q.token_stride + (n.h * G + row - j * G) * a.q.head_stride;
    };
    for (int which = 0; more; which ^= 1) {
        const int h = s_item[which].h, row0 = s_item[which].row0, rows = s_item[which].rows;
        const int tok0 = s_item[which].tok0, tok1 = s_item[which].tok1, before = s_item[which].len - s_item[which].n;
        const int* const table = a.table + s_item[which].b * a.table_stride;
        // Stages begin at multiples of 16 tokens, so that they lie in one page where pages are such multiples.
        const int base0 = tok0 & ~15, count = tok1 - base0 - group * S::kTokens;
        const int stages = count <= 0 ? 0 : (count + S::kGroups * S::kTokens - 1) / (S::kGroups * S::kTokens);

        // ---- page ids of the first stages: lane l knows token l of a stage
        auto token_of = [&](int i) { return base0 + (i * S::kGroups + group) * S::kTokens + (lane & (S::kTokens - 1)); };
        auto page_of = [&](int i) {  // page id of the lane's token, −1 outside the piece
            const int tok = token_of(i);
            return tok >= tok0 && tok < tok1 ? __ldg(table + sp.page_index(tok)) : -1;
        };
        int first[S::kAhead];
#pragma unroll
        for (int i = 0; i < S::kAhead; ++i) first[i] = page_of(i);

        // ---- queries of the thread's rows g and g + 8, asked for ahead of the tokens' bytes
        uint32_t q[Q8 ? 1 : KS][4];
        int see_lo[2], see_hi[2];   // tokens that a row sees
        uint2 raw[Q8 ? 2 : 1][Q8 ? KS : 1];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = row0 + rw * 16 + g + 8 * x, j = sp.over_G(r);
            const bool live = r < rows;
            see_hi[x] = live ? before + j + 1 : 0x7fffffff;
            see_lo[x] = live && a.window > 0 ? static_cast<int>(max(0ll, static_cast<long long>(see_hi[x]) - a.window)) : 0;
            const __nv_bfloat16* src = live ? query_row(s_item[which], r) : a.q.data;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                if (!Q8) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int k = ks * 16 + 2 * t4 + 8 * y;
                        q[Q8 ? 0 : ks][x + 2 * y] = live && k < a.head_dim ? *reinterpret_cast<const uint32_t*>(src + k) : 0u;
                    }
                } else {
                    // four values in a row for each k-step and lane, like the keys' codes below
                    const int k = (ks >> 2) * 64 + t4 * 16 + (ks & 3) * 4;
                    raw[Q8 ? x : 0][Q8 ? ks : 0] = live && k < a.head_dim ? *reinterpret_cast<const uint2*>(src + k) : make_uint2(0, 0);
                }
            }
        }

        // ---- loads
        // Scales of the lane's token travel by register until the stage before theirs has been used (for an iteration
        // and a half where kSlots is even), then through shared memory.  As they come: a conversion right behind the
        // load would wait for it in every stage (80 µs for 74 at 64 ragged requests).
        struct Scales {
            __nv_bfloat16 k, v;
        };
        const Scales none = {__ushort_as_bfloat16(0), __ushort_as_bfloat16(0)};
        Scales found = none, older = none;
        auto put_scales = [&](const Scales& x, int stage) {
            if (Q8 && stage < stages && rw == 0 && lane < S::kTokens) {
                const float v = __bfloat162float(x.v);
                scales[stage % S::kScaleSlots * S::kTokens + lane] = make_float2(__bfloat162float(x.k), __log2f(v < kLeastScale ? kLeastScale : v));
            }
        };
        long long off = -1;     // of the lane's token, in the stage whose keys were asked for last; −1: none
        long long off0[S::kSub];  // of the first token of each 16
        bool even = false;      // the tokens are all there, those of a 16 token_stride apart, with rows of D values
        auto find = [&](int i, int page) {  // stage i
            const int tok = token_of(i);
            const int pi = sp.page_index(tok);
            const int in_page = tok - pi * a.page_size;
            off = -1;
            if (i < stages && tok >= tok0 && tok < tok1) {
                if (page >= 0 && page < a.pages)
                    off = page * a.page_stride + in_page * a.token_stride + h * a.head_stride;
                else
                    record_status(a.status, kStatusInvalid);
            }
            if (Q8) {
                found = none;
                if (off >= 0) {
                    const long long s = (static_cast<long long>(page) * a.kv_heads + h) * a.page_size + in_page;
                    found.k = a.k_scales[s];
                    found.v = a.v_scales[s];
                }
            }
#pragma unroll
            for (int sub = 0; sub < S::kSub; ++sub) off0[sub] = __shfl_sync(~0u, off, 16 * sub);
            const long long mine = S::kSub == 2 && (lane & 16) ? off0[S::kSub - 1] : off0[0];
            even = __all_sync(~0u, mine >= 0 && off == mine + (lane & 15) * a.token_stride) && d_chunks == S::kChunks;
        };
        auto load = [&](auto key, int slot, bool any) {  // keys or values of the stage found last
            constexpr bool KEY = decltype(key)::value;
            if (any) {
                // place of (load_r, load_c); rows p further on keep it but for the turn of p's low bits
                const uint32_t dst = ring + slot * S::kHalf + load_r * kRow + ((load_c ^ turn<kRow, Q8, KEY>(load_r)) << 4);
                const uint8_t* src = static_cast<const uint8_t*>(KEY ? a.k : a.v);
                auto to = [&](int p) { return (dst ^ (turn<kRow, Q8, KEY>(p) << 4)) + p * kRow; };
                if (even) {
                    // (a pass may reach into the second 16 tokens)
                    const uint8_t* from = src + (kPerPass > 16 && load_r >= 16 ? off0[S::kSub - 1] : off0[0]) * S::kElt +
                                          (load_r & 15) * a.token_stride * S::kElt + load_c * 16;
#pragma unroll
                    for (int p = 0; p < S::kTokens; p += kPerPass) {
                        if (S::kSub == 2 && p == 16)
                            from = src + off0[S::kSub - 1] * S::kElt + load_r * a.token_stride * S::kElt + load_c * 16;
                        cp_async16(to(p), from);
                        from += kPerPass * S::kElt * a.token_stride;
                    }
                } else {
#pragma unroll
                    for (int p = 0; p < S::kTokens; p += kPerPass) {
                        const long long o = __shfl_sync(~0u, off, (p + load_r) & 31);
                        const bool there = o >= 0 && load_c < d_chunks;
                        const uint8_t* from = src + (there ? o * S::kElt + load_c * 16 : 0);
                        cp_async16_zfill(to(p), from, there ? 16 : 0);
                    }
                }
            }
            cp_async_commit();
        };
        // Copy n holds the keys (n even) or values of stage n / 2; copy n + kSlots − 1 is asked for when copy n is
        // there, into the slot of copy n − 1.  So stage i + kSlots / 2 is found while stage i is worked on.
        auto load_next = [&](auto key, int i, int slot, int& page, int n) {
            if (decltype(key)::value) {
                find(i + S::kSlots / 2, page);
                page = page_of(i + S::kSlots / 2 + 1);
            }
            load(key, slot, (n >> 1) < stages);
        };
        constexpr bool kOdd = S::kSlots % 2 != 0;
        using First = std::integral_constant<bool, kOdd>;    // keys where kSlots is odd: copy 2i + kSlots − 1
        using Second = std::integral_constant<bool, !kOdd>;  // copy 2i + kSlots
        Scales begin[S::kAhead];
#pragma unroll
        for (int n = 0; n < S::kSlots - 1; ++n) {
            if ((n & 1) == 0) {
                find(n >> 1, first[n >> 1]);
                begin[n >> 1] = found;
                load(std::true_type(), n, (n >> 1) < stages);
            } else {
                load(std::false_type(), n, (n >> 1) < stages);
            }
        }
        int page_next = page_of(S::kSlots / 2);

        float row_scale[2] = {sp.scale_log2, sp.scale_log2};  // of scores, to base 2
        if (!Q8) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int x = 0; x < 4; ++x) q[Q8 ? 0 : ks][x] ^= sp.flip;
        } else {
            // As fp16, after a multiplication of the row by a power of two that takes its largest value to 2¹⁴ and more:
            // values down to 2⁻³¹ of it keep all bits, smaller ones err by 2⁻³⁹ of it (by nothing where the row is below
            // 2⁻⁹⁵: a bf16 is a multiple of 2⁻¹³³).
            float to16[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float most = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint2 w = raw[Q8 ? x : 0][Q8 ? ks : 0];
                    most = fmaxf(most, fmaxf(fmaxf(fabsf(bf16_lo(w.x)), fabsf(bf16_hi(w.x))), fmaxf(fabsf(bf16_lo(w.y)), fabsf(bf16_hi(w.y)))));
                }
                most = quad_max(most);
                const int e = min(max(static_cast<int>(__float_as_uint(most) >> 23), 32), 254) - 127;
                to16[x] = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
                row_scale[x] *= __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
            }
            if (group == 0)  // the other groups have the same rows
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const uint2 u = raw[0][Q8 ? ks : 0], w = raw[Q8 ? 1 : 0][Q8 ? ks : 0];
                    queries[(rw * KS + ks) * 32 + lane] =
                        make_uint4(pack_f16(bf16_lo(u.x) * to16[0], bf16_hi(u.x) * to16[0]) ^ sp.flip, pack_f16(bf16_lo(w.x) * to16[1], bf16_hi(w.x) * to16[1]) ^ sp.flip,
                                   pack_f16(bf16_lo(u.y) * to16[0], bf16_hi(u.y) * to16[0]) ^ sp.flip, pack_f16(bf16_lo(w.y) * to16[1], bf16_hi(w.y) * to16[1]) ^ sp.flip);
                }
            __syncthreads();
        }
        // Tokens before all_hi and from all_lo on are seen by every row of the warp.
        int all_hi, all_lo;
        {
            const int j0 = sp.over_G(row0 + rw * 16), j1 = sp.over_G(max(min(row0 + rw * 16 + 15, rows - 1), 0));
            all_hi = before + j0 + 1;
            all_lo = a.window > 0 ? static_cast<int>(max(0ll, static_cast<long long>(before) + j1 + 1 - a.window)) : 0;
        }

        // ---- the next item, and its first page ids and its queries to L2, while this one's first bytes are on their way
        if (warp == 0) {
            if (lane == 0) s_more = s_walk.next(sp, s_item[which ^ 1]);
            __syncwarp();
            if (s_more) {
                const Item& n = s_item[which ^ 1];
                const int tok = n.tok0 + lane * 32;  // a line of 32 page ids, or fewer where pages hold several tokens
                if (lane < S::kAhead * S::kGroups * S::kTokens / 32 && tok < n.tok1)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.table + n.b * a.table_stride + sp.page_index(tok)));
                for (int x = lane; x < 16 * R * 4; x += 32)
                    if (n.row0 + (x >> 2) < n.rows && 64 * (x & 3) < a.head_dim)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(query_row(n, n.row0 + (x >> 2)) + 64 * (x & 3)));
            }
        }

        float o[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i][x] = 0.f;
        // Format 16: the reference score, unscaled, and the sum of the weights 2^(row_scale · (s − m)).
        // Format 8: the reference of score + log2(value scale), to base 2: the weights times their value scales are
        // near 2⁷ whatever the scales (the reference is taken 7 lower); the sum is that of the weights by the same
        // reference, over 2⁷.
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

#pragma unroll
        for (int i = 0; i < S::kSlots / 2; ++i) put_scales(begin[i], i);
        int get = 0;
        for (int i = 0; i < stages; ++i) {
            cp_async_wait<S::kSlots - 2>();
            if (!kOdd) {
                if (i > 1) put_scales(older, i + S::kSlots / 2 - 2);
                older = found;
            }
            group_sync<R>(group);
            load_next(First(), i, get == 0 ? S::kSlots - 1 : get - 1, page_next, 2 * i + S::kSlots - 1);
            const int base = base0 + (i * S::kGroups + group) * S::kTokens;
            const int key_slot = get;
            const uint32_t keys = ring + get * S::kHalf;
            if (++get == S::kSlots) get = 0;
            const uint32_t vals = ring + get * S::kHalf;
            if (++get == S::kSlots) get = 0;
            const float2* stage_scales = scales + i % S::kScaleSlots * S::kTokens;

            // ---- scores: s[2·sub + nt][x] of row g + 8·(x >> 1), token 16·sub + 8·nt + 2·t4 + (x & 1)
            float s[2 * S::kSub][4];
#pragma unroll
            for (int y = 0; y < 2 * S::kSub; ++y)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[y][x] = 0.f;
            if (!Q8) {
                // token (lane >> 4) · 8 + (lane & 7), chunk 2·ks + ((lane >> 3) & 1)
                const uint32_t from = keys + ((lane >> 4) * 8 + (lane & 7)) * kRow + ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int sub = 0; sub < S::kSub; ++sub) {
                        uint32_t k[4];
                        ldmatrix_x4((from ^ ((ks & 3) << 5)) + (ks >> 2) * 128 + sub * 16 * kRow, k);
                        mma16816<false>(s[2 * sub], q[Q8 ? 0 : ks], k[0], k[1]);
                        mma16816<false>(s[2 * sub + 1], q[Q8 ? 0 : ks], k[2], k[3]);
                    }
            } else {
                // token 8·y + g, chunk 4·kb + t4: four k-steps of two pairs
                const uint32_t from = keys + g * kRow + ((t4 ^ turn<kRow, Q8, true>(g)) << 4);
#pragma unroll
                for (int kb = 0; kb < KS / 4; ++kb) {
                    uint32_t w[2 * S::kSub][4];
#pragma unroll
                    for (int y = 0; y < 2 * S::kSub; ++y) {
                        const uint4 v = lds128((from ^ ((kb & 1) << 6)) + (kb >> 1) * 128 + y * 8 * kRow);
                        w[y][0] = v.x ^ 0x80808080u, w[y][1] = v.y ^ 0x80808080u, w[y][2] = v.z ^ 0x80808080u, w[y][3] = v.w ^ 0x80808080u;
                    }
                    // (neighbouring products go to different sums)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint4 v = queries[(rw * KS + kb * 4 + x) * 32 + lane];
                        const uint32_t f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int y = 0; y < 2 * S::kSub; ++y)
                            mma16816<true>(s[y], f, codes_f16(w[y][x], 0x4140), codes_f16(w[y][x], 0x4342));
                    }
                }
            }
            if (Q8) {
#pragma unroll
                for (int y = 0; y < 2 * S::kSub; ++y) {
                    const float4 f = *reinterpret_cast<const float4*>(stage_scales + y * 8 + 2 * t4);
                    s[y][0] = fmaf(s[y][0], row_scale[0] * f.x, f.y);
                    s[y][1] = fmaf(s[y][1], row_scale[0] * f.z, f.w);
                    s[y][2] = fmaf(s[y][2], row_scale[1] * f.x, f.y);
                    s[y][3] = fmaf(s[y][3], row_scale[1] * f.z, f.w);
                }
            }
            // Some row does not see some token of the stage; there are such tokens, too, past the end.
            const bool hidden = min(base + S::kTokens, tok1) > all_hi || base < all_lo;
            const bool partly = hidden || base + S::kTokens > tok1 || base < tok0;
            if (partly) {
#pragma unroll
                for (int y = 0; y < 2 * S::kSub; ++y)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int tok = base + y * 8 + 2 * t4 + (x & 1);
                        if (tok >= min(see_hi[x >> 1], tok1) || tok < max(see_lo[x >> 1], tok0)) s[y][x] = -INFINITY;
                    }
            }

            // ---- reference
            float grown[2] = {m[0], m[1]};
#pragma unroll
            for (int y = 0; y < 2 * S::kSub; ++y)
#pragma unroll
                for (int x = 0; x < 4; ++x) grown[x >> 1] = fmaxf(grown[x >> 1], s[y][x]);
            grown[0] = quad_max(grown[0]);
            grown[1] = quad_max(grown[1]);
            const float by0 = (grown[0] - m[0]) * (Q8 ? 1.f : row_scale[0]), by1 = (grown[1] - m[1]) * (Q8 ? 1.f : row_scale[1]);
            constexpr float kFar = Q8 ? kLift + 8.f : 8.f;
            if (__any_sync(~0u, by0 > kFar || by1 > kFar)) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (Q8) grown[x] = fmaxf(m[x], grown[x] - kLift);
                    const float keep = m[x] == -INFINITY ? 0.f : ex2(Q8 ? m[x] - grown[x] : x ? -by1 : -by0);
                    l[x] = fminf(l[x], 3e38f) * keep;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        o[n][2 * x] *= keep;
                        o[n][2 * x + 1] *= keep;
                    }
                    m[x] = grown[x];
                }
            }
            // ---- weights
            const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0] * (Q8 ? 1.f : row_scale[0]),
                                  m[1] == -INFINITY ? 0.f : m[1] * (Q8 ? 1.f : row_scale[1])};
#pragma unroll
            for (int y = 0; y < 2 * S::kSub; ++y) {
                // 1 / value scale of the lane's tokens, over 2⁷: a number even where the scale is none, since a hidden
                // token's weight of 0 makes it 0 then.
                float inv[2] = {1.f, 1.f};
                if (Q8) {
                    const float4 f = *reinterpret_cast<const float4*>(stage_scales + y * 8 + 2 * t4);
                    inv[0] = fminf(ex2(-f.y), 3e38f) * kLower;
                    inv[1] = fminf(ex2(-f.w), 3e38f) * kLower;
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (Q8) {
                        s[y][x] = ex2(s[y][x] - ref[x >> 1]);
                        l[x >> 1] = fmaf(s[y][x], inv[x & 1], l[x >> 1]);
                    } else {
                        s[y][x] = ex2(fmaf(s[y][x], row_scale[x >> 1], -ref[x >> 1]));
                        l[x >> 1] += s[y][x];
                    }
                }
            }

            // ---- values
            cp_async_wait<S::kSlots - 2>();
            group_sync<R>(group);
            load_next(Second(), i, key_slot, page_next, 2 * i + S::kSlots);
            if (!Q8) {
                bool odd = false;  // a value that is not finite, in tokens that some rows do not see
                if (hidden) {
                    for (int x = lane; x < S::kTokens * S::kChunks; x += 32) {
                        const uint4 w = lds128(vals + x * 16);
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            odd |= (u[y] & 0x7F80u) == 0x7F80u || (u[y] & 0x7F800000u) == 0x7F800000u;
                    }
                }
                if (__any_sync(~0u, odd)) {
                    // 0 · ∞ would spoil the rows that do not see the token: add token by token to those that do.
                    for (int tk = 0; tk < S::kTokens; ++tk) {
                        const int from = (lane & ~3) | ((tk & 7) >> 1);
                        float p[2];
                        bool seen[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            float v = 0.f;
#pragma unroll
                            for (int y = 0; y < 2 * S::kSub; ++y)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (y == tk >> 3 && e == (tk & 1)) v = s[y][2 * x + e];
                            p[x] = __shfl_sync(~0u, v, from);
                            seen[x] = base + tk < min(see_hi[x], tok1) && base + tk >= max(see_lo[x], tok0);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint32_t w;
                            asm volatile("ld.shared.u32 %0, [%1];"
                                         : "=r"(w)
                                         : "r"(vals + tk * kRow + ((n ^ turn<kRow, Q8, false>(tk)) << 4) + 4 * t4));
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                if (seen[x]) {
                                    o[n][2 * x] += p[x] * bf16_lo(w);
                                    o[n][2 * x + 1] += p[x] * bf16_hi(w);
                                }
                        }
                    }
                } else {
                    // The weights as two bf16 each (16 bits): one alone would err as much as the result's rounding.
                    uint32_t hi[S::kSub][4], lo[S::kSub][4];
#pragma unroll
                    for (int sub = 0; sub < S::kSub; ++sub)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const float p0 = s[2 * sub + (x >> 1)][2 * (x & 1)], p1 = s[2 * sub + (x >> 1)][2 * (x & 1) + 1];
                            hi[sub][x] = pack_bf16(p0, p1);
                            lo[sub][x] = pack_bf16(p0 - bf16_lo(hi[sub][x]), p1 - bf16_hi(hi[sub][x]));
                        }
                    // token ((lane >> 3) & 1) · 8 + (lane & 7), chunk 2·n + (lane >> 4)
                    const uint32_t from = vals + (((lane >> 3) & 1) * 8 + (lane & 7)) * kRow + (((lane >> 4) ^ (lane & 7)) << 4);
#pragma unroll
                    for (int n = 0; n < NT / 2; ++n)
#pragma unroll
                        for (int sub = 0; sub < S::kSub; ++sub) {
                            uint32_t v[4];
                            ldmatrix_x4_trans((from ^ ((n & 3) << 5)) + (n >> 2) * 128 + sub * 16 * kRow, v);
                            mma16816<false>(o[2 * n], hi[sub], v[0], v[1]);
                            mma16816<false>(o[2 * n + 1], hi[sub], v[2], v[3]);
                            mma16816<false>(o[2 * n], lo[sub], v[0], v[1]);
                            mma16816<false>(o[2 * n + 1], lo[sub], v[2], v[3]);
                        }
                }
            } else {
                // Weights times value scales as fp16 (2⁻¹¹): an eighth of the result's rounding.  Below 2⁻²¹ of the
                // reference they err by 2⁻³² of it, which shows only where the tokens above have codes of zero.
#pragma unroll
                for (int sub = 0; sub < S::kSub; ++sub) {
                    uint32_t p[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        p[x] = pack_f16(s[2 * sub + (x >> 1)][2 * (x & 1)], s[2 * sub + (x >> 1)][2 * (x & 1) + 1]);
                    // Column n of output tile i is value 16·n + i (8·n + i for D = 64) of the row's 128: a lane's
                    // 16 (8) bytes of a token row are its column of 16 (8) tiles.
                    constexpr int kBytes = D == 64 ? 8 : 16;
                    const int chunk = D == 64 ? g >> 1 : g;
                    const uint32_t from = vals + 2 * t4 * kRow + ((chunk ^ turn<kRow, Q8, false>(2 * t4)) << 4) + (D == 64 ? 8 * (g & 1) : 0);
#pragma unroll
                    for (int hb = 0; hb < NT / kBytes; ++hb) {
                        uint32_t w[4][kBytes / 4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {  // token 16·sub + 2·t4 + (x & 1) + 8·(x >> 1)
                            const int r = (x & 1) + 8 * (x >> 1);
                            const uint32_t at = (from ^ (turn<kRow, Q8, false>(r & 1) << 4)) + (sub * 16 + r) * kRow + hb * 128;
                            if (kBytes == 16) {
                                const uint4 v = lds128(at);
                                w[x][0] = v.x ^ 0x80808080u;
                                w[x][1] = v.y ^ 0x80808080u;
                                w[x][kBytes / 4 - 2] = v.z ^ 0x80808080u;
                                w[x][kBytes / 4 - 1] = v.w ^ 0x80808080u;
                            } else {
                                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[x][0]), "=r"(w[x][1]) : "r"(at));
                                w[x][0] ^= 0x80808080u;
                                w[x][1] ^= 0x80808080u;
                            }
                        }
#pragma unroll
                        for (int y = 0; y < kBytes / 4; ++y) {
                            // bytes of two tokens side by side: (a0 b0 a1 b1), (a2 b2 a3 b3)
                            const uint32_t e0 = __byte_perm(w[0][y], w[1][y], 0x5140), e1 = __byte_perm(w[0][y], w[1][y], 0x7362);
                            const uint32_t f0 = __byte_perm(w[2][y], w[3][y], 0x5140), f1 = __byte_perm(w[2][y], w[3][y], 0x7362);
                            mma16816<true>(o[hb * 16 + 4 * y], p, codes_f16(e0, 0x4140), codes_f16(f0, 0x4140));
                            mma16816<true>(o[hb * 16 + 4 * y + 1], p, codes_f16(e0, 0x4342), codes_f16(f0, 0x4342));
                            mma16816<true>(o[hb * 16 + 4 * y + 2], p, codes_f16(e1, 0x4140), codes_f16(f1, 0x4140));
                            mma16816<true>(o[hb * 16 + 4 * y + 3], p, codes_f16(e1, 0x4342), codes_f16(f1, 0x4342));
                        }
                    }
                }
            }
        }
        cp_async_wait<0>();

        // ---- the groups' sums meet in shared memory: [warp][16 rows][kMeetRow], then the reference and sum of each row
        __syncthreads();
        float* s_o = reinterpret_cast<float*>(smem);
        float* s_stat = s_o + kWarps * 16 * S::kMeetRow;  // [2][warp][16]
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            l[x] = quad_sum(l[x]);
            if (t4 == 0) {
                s_stat[warp * 16 + g + 8 * x] = m[x] * (Q8 ? 1.f : row_scale[x]);
                s_stat[kWarps * 16 + warp * 16 + g + 8 * x] = fminf(l[x], 3e38f);
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float* to = s_o + (warp * 16 + g + 8 * x) * S::kMeetRow;
            if (!Q8) {
#pragma unroll
                for (int n = 0; n < NT; ++n) *reinterpret_cast<float2*>(to + n * 8 + 2 * t4) = make_float2(o[n][2 * x], o[n][2 * x + 1]);
            } else {
                constexpr int kRun = D == 64 ? 8 : 16;  // neighbouring values of a lane's column
#pragma unroll
                for (int n = 0; n < NT; n += 4)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float4*>(to + n / kRun * 128 + (2 * t4 + e) * kRun + n % kRun) =
                            make_float4(o[n][2 * x + e], o[n + 1][2 * x + e], o[n + 2][2 * x + e], o[n + 3][2 * x + e]);
            }
        }
        __syncthreads();

        const Item it = s_item[which];
        const bool whole = it.whole();
        more = s_more;
        const Parts<16 * R, D> parts(sp, s_walk, it, kFixed);
        float* const part = parts.at(static_cast<int>(blockIdx.x) - parts.first);
        for (int x = tid; x < 16 * R * (D / 4); x += kThreads) {
            const int r = x / (D / 4), col = x % (D / 4) * 4, row = row0 + r;
            if (row >= rows || col >= a.head_dim) continue;
            float mm = -INFINITY;
#pragma unroll
            for (int k = 0; k < S::kGroups; ++k) mm = fmaxf(mm, s_stat[k * R * 16 + r]);
            const float rm = mm == -INFINITY ? 0.f : mm;
            float ll = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < S::kGroups; ++k) {
                const float f = ex2(s_stat[k * R * 16 + r] - rm);
                const float4 w = *reinterpret_cast<const float4*>(s_o + (k * R * 16 + r) * S::kMeetRow + col);
                const float fv = Q8 ? f * kLower : f;
                ll += f * s_stat[kWarps * 16 + k * R * 16 + r];
                v[0] += fv * w.x, v[1] += fv * w.y, v[2] += fv * w.z, v[3] += fv * w.w;
            }
            if (whole) {
                put_row(sp, it, row, col, v, 4, ll);
            } else {
                if (col == 0) {
                    part[r] = mm;
                    part[16 * R + r] = fminf(ll, 3e38f);
                }
                *reinterpret_cast<float4*>(part + 32 * R + r * D + col) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
        __syncthreads();
        if (!whole)
            parts.finish(sp, s_last, [] { __syncthreads(); }, [&](int k0, int n, int step, bool last) {
                if (n <= 4)
                    parts.template join_rows<kWarps, 4>(sp, it, warp, lane, k0, n, step, last);
                else
                    parts.template join_rows<kWarps, 16>(sp, it, warp, lane, k0, n, step, last);
            });
    }
}

int dim_of(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

// Query rows to a key-value head of a request, on the average.
int64_t average_rows(int32_t B, int64_t T, int G) { return (T + B - 1) / B * G; }

// Whether the tensor-core kernel takes the call.  A row tile of 16 or 32 rows
// is a pass over the request's tokens here, one of 128 rows there, but a piece
// of work starts and joins in less time here.  µs here and there, requests of
// 1024 to 8192 tokens (16 of them) where nothing else is said:
// head_dim 128, 16 rows: 56 and 67; 24: 67 and 67, and 21 and 28 for 64 requests
// of 128 tokens; 32: 71 and 66; 40: 108 and 68.  64, 32 rows: 26 and 29; 40: 35
// and 29.  256, 32 rows: 69 and 90; 52, for 64 requests of 512 tokens: 66 and 56.
// Format 8: head_dim 128, 40 rows: 81 and 94; 64: 103 and 94; 104: 166 and 97.
// 256, 52 rows: 110 and 112.  64, 64 rows: 27 and 33; 104: 39 and 34.
// Where requests × heads leave half of the 152 SMs without an item of their own,
// that kernel joins many large parts: head_dim 256, 52 rows, 4 heads, 4 requests
// of 512 tokens 28 and 44, of 2048 tokens 34 and 62; in format 8 22 and 48, 31
// and 67; 64, 104 rows, 2 heads, 4 requests of 2048 tokens in format 8: 14 and 25.
bool many_rows(int32_t B, int64_t T, int G, int32_t kv_heads, int D, bool q8) {
    const int limit = q8 ? (D == 64 ? 64 : 48) : D == 128 ? 24 : 32;
    const bool few = static_cast<int64_t>(B) * kv_heads < 76 && (q8 || D == 256);
    return average_rows(B, T, G) > (few ? 2 * limit : limit);
}

// Warps (of 16 rows) that share a stage.  With two, 17 to 32 rows are one pass
// over the cache instead of two: 69 and 475 µs for 76 and 932 at head_dim 256,
// 32 rows, in the two calls above, but 243 for 301 only where 64 is the
// head_dim (and 54 for 52 where 8 rows are all there are: fewer rings, and a
// barrier of two warps).  Format 8 is bound by its decoding, which each row
// tile repeats in any case: 61 µs with one and 65 with two warps at 32 rows,
// 570 and 545 in longer requests.
int row_warps(int32_t B, int64_t T, int G, bool q8) { return !q8 && average_rows(B, T, G) > 16 ? 2 : 1; }

template <int D, bool Q8, int R>
cudaError_t run(const SplitArgs& sp, const DeviceInfo& dev, cudaStream_t stream) {
    using S = Shape<D, Q8, R>;
    // CTAs that an SM holds, asked once per device.
    static std::atomic<int> known[kMaxDevices];
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err != cudaSuccess) return err;
    int per_sm = known[device & (kMaxDevices - 1)].load(std::memory_order_relaxed);
    if (per_sm == 0) {
        err = cudaFuncSetAttribute(attn_split_kernel<D, Q8, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (err != cudaSuccess) return err;
        err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, attn_split_kernel<D, Q8, R>, kThreads, S::kSmem);
        if (err != cudaSuccess) return err;
        if (per_sm < 1) return cudaErrorInvalidConfiguration;
        known[device & (kMaxDevices - 1)].store(per_sm, std::memory_order_relaxed);
    }
    // At least as many units as the batch can have: a CTA for each, where they are few.
    const AttnArgs& a = sp.a;
    const double reach = std::min(static_cast<double>(a.width) * a.page_size, a.window > 0 ? static_cast<double>(a.window) + a.T : 1e18);
    const double most = static_cast<double>(a.kv_heads) * (a.B + static_cast<double>(a.T) * sp.G / (16 * R)) * (reach / kTile + 2 + S::kFixed);
    const int grid = static_cast<int>(std::min<double>(std::min(per_sm * dev.sm_count, kMaxCtas), most));
    attn_split_kernel<D, Q8, R><<<grid, kThreads, S::kSmem, stream>>>(sp);
    return cudaGetLastError();
}

template <int D, bool Q8>
cudaError_t run_rows(const SplitArgs& sp, const DeviceInfo& dev, cudaStream_t stream) {
    if constexpr (!Q8)
        if (row_warps(sp.a.B, sp.a.T, sp.G, Q8) == 2) return run<D, Q8, 2>(sp, dev, stream);
    return run<D, Q8, 1>(sp, dev, stream);
}

template <bool Q8>
cudaError_t run_dim(const SplitArgs& sp, const DeviceInfo& dev, cudaStream_t stream) {
    const int D = dim_of(sp.a.head_dim);
    if (D == 64) return run_rows<64, Q8>(sp, dev, stream);
    if (D == 128) return run_rows<128, Q8>(sp, dev, stream);
    return run_rows<256, Q8>(sp, dev, stream);
}

}  // namespace

size_t attn_decode_workspace_bytes(int32_t B, int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim, bool q8) {
    const int G = q_heads / kv_heads, D = dim_of(head_dim);
    if (B <= 0) B = 1;
    const bool many = many_rows(B, T, G, kv_heads, D, q8);
    const size_t part = many ? attn_tc_partial_floats(head_dim) : partial_floats(16 * row_warps(B, T, G, q8), D);
    return 2 * (kMaxCtas * sizeof(unsigned long long) + (many ? kMaxTcCtas : kMaxCtas) * part * sizeof(float));
}

cudaError_t launch_attn_decode(AttnArgs a, bool q8, void* workspace, const DeviceInfo& dev, cudaStream_t stream) {
    divide_by(a.page_size, &a.page_mul, &a.page_shift);
    SplitArgs sp = {};
    sp.a = a;
    sp.arrived = static_cast<unsigned long long*>(workspace);
    sp.partial = reinterpret_cast<float*>(sp.arrived + 2 * kMaxCtas);
    sp.G = a.q_heads / a.kv_heads;
    divide_by(sp.G, &sp.G_mul, &sp.G_shift);
    sp.rows_each = static_cast<int>(a.T / a.B);
    // A factor below zero turns the queries' signs over, and one of zero is one so small that every weight is 1: the
    // largest score is then that of the unscaled products, and hidden ones stay at −∞.
    sp.scale_log2 = std::max(std::fabs(a.scale) * 1.4426950408889634f, 1e-30f);
    sp.flip = a.scale < 0.f ? 0x80008000u : 0u;
    if (many_rows(a.B, a.T, sp.G, a.kv_heads, dim_of(a.head_dim), q8)) return launch_attn_tc(sp, q8, dev, stream);
    return q8 ? run_dim<true>(sp, dev, stream) : run_dim<false>(sp, dev, stream);
}

}  // namespace w4
