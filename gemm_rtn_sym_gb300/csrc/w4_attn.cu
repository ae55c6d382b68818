// Attention of the newest tokens of each request over its pages of the
// key-value cache.
//
// For a row at position p: o = Σ_t 2^(s_t − m) v_t / Σ_t 2^(s_t − m) over the
// tokens it sees, s_t = scale · log2(e) · q·k_t and m the largest s_t, in one
// pass over the tokens: where the running maximum grows from m to m', sums and
// values so far are multiplied by 2^(m − m').
//
// Every byte of keys and values is used for a few rows only (query heads per
// key-value head × new tokens), so the pass is bound by reading the cache.
// The work is the list of all (request, key-value head, row tile, 64 tokens),
// in that order, cut into equal runs, one for each CTA of a grid that is
// resident at once: requests of any lengths load every SM alike.  A run's
// first and last items may belong to several CTAs; those leave their sums in
// the workspace, and a second small kernel joins them.
//
// Inside a CTA each group of R warps (16 query rows each) streams its own
// tokens through its own ring of cp.async copies, keys and values in turn, so
// that no barrier of the whole CTA stands in the loop; products run on m16n8k16 MMAs from registers,
// rows (at most 16·R) as their M, padded with zeros.
#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "w4_device.cuh"
#include "w4_kv.h"

namespace w4 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 64;       // tokens of a work item
constexpr int kFixed = 3;       // an item's fixed cost (its first loads' latency, its sums' way out), in tiles
constexpr int kMaxLength = 0x7fff0000;  // token numbers a little past a length stay below 2³¹
constexpr int kMaxDevices = 64;  // as many as the library knows (device_info refuses others)
constexpr int kMaxCtas = 1024;  // largest grid: bounds the workspace

// What the join needs to know of a CTA's last item where other CTAs carry it on.
struct Carried {
    int last;     // last CTA of the item; −1: no item of this CTA is carried on
    int head;     // key-value head
    int row0;     // first row of the row tile
    int rows;     // rows of the request (new tokens × query heads per key-value head)
    int start;    // first token row of the request
    int before;   // tokens before the new ones (may be negative)
};

// Largest score, largest weight's exponent (score + log2 of the value's scale),
// sum: 16·R of each, then 16·R rows of D values.
__host__ __device__ constexpr size_t partial_floats(int R, int D) { return static_cast<size_t>(16 * R) * (3 + D); }

struct SplitArgs {
    AttnArgs a;
    Carried* carried;   // [grid]
    float* partial;     // [grid][2][partial_floats]
    float scale_log2;
};

// ------------------------------------------------------------- small pieces
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
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

// --------------------------------------------------------------- work list
// A request's part of the work: rows and tokens, clipped to what is there.
struct Request {
    int start, n;     // token rows
    int len;          // tokens in the cache
    int low;          // first token that any row sees
    int tiles;        // 64-token tiles from the one of `low`
    int row_tiles;
};

__device__ __forceinline__ Request request(const AttnArgs& a, int b, int rows_per_tile) {
    Request r;
    if (a.starts) {
        const long long T = a.T;
        const long long s = min(max(static_cast<long long>(a.starts[b]), 0ll), T);
        const long long e = min(max(static_cast<long long>(a.starts[b + 1]), s), T);
        r.start = static_cast<int>(s);
        r.n = static_cast<int>(e - s);
    } else {
        r.n = static_cast<int>(a.T / a.B);
        r.start = b * r.n;
    }
    const long long most = min(static_cast<long long>(a.width) * a.page_size, static_cast<long long>(kMaxLength));
    const int len = a.lens[b];
    if (len < 0 || len > most) record_status(a.status, kStatusInvalid);
    r.len = len < 0 ? 0 : static_cast<int>(min(static_cast<long long>(len), most));
    const long long low = a.window > 0 ? static_cast<long long>(r.len) - r.n - a.window + 1 : 0;
    r.low = static_cast<int>(max(low, 0ll));
    const int rows = r.n * (a.q_heads / a.kv_heads);
    // A request without tokens still has its rows of zeros to write: one tile.
    r.tiles = max(1, (r.len + kTile - 1) / kTile - r.low / kTile);
    r.row_tiles = (rows + rows_per_tile - 1) / rows_per_tile;
    return r;
}

// Units of work of a request: each item (head, row tile) counts kFixed units
// and then one for each of its tiles.
__device__ __forceinline__ long long units(const AttnArgs& a, const Request& r) {
    return static_cast<long long>(a.kv_heads) * r.row_tiles * (r.tiles + kFixed);
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
    static constexpr int kHalf = kTokens * kRow;     // a slot of the ring: a stage's keys or values
    // Three CTAs of 168 registers on an SM, where the outputs' D / 2 leave that; else two.
    static constexpr int kCtas = D == 256 ? 2 : 3;
    static constexpr int kBudget = (kCtas == 3 ? 72 : 108) * 1024;
    static constexpr int kFit = kBudget / (kGroups * (kHalf + (Q8 ? kTokens * 8 : 0)));
    static constexpr int kSlots = kFit > 12 ? 12 : kFit;
    static constexpr int kAhead = (kSlots + 1) / 2;  // stages whose keys may be under way or in use
    static constexpr int kRing = kSlots * kHalf;
    // (key scale, log2 of value scale) of each token, for the stages on the way and the one in use
    static constexpr int kScaleSlots = kAhead + 1;
    static constexpr int kScales = Q8 ? kScaleSlots * kTokens * 8 : 0;
    static constexpr int kGroup = kRing + kScales;
    static constexpr int kMerge = kWarps * 16 * (D + 3) * 4;
    static constexpr int kSmem = kGroups * kGroup > kMerge ? kGroups * kGroup : kMerge;
    static_assert(kSlots >= 3, "a slot in use, two on the way");
};

// Where 16-byte chunk c of token row r lies in a stage's keys (KEY) or values:
// the loads of eight lanes that a shared-memory access serves at once fall in
// different banks.
template <int D, bool Q8, bool KEY>
__device__ __forceinline__ uint32_t place(int r, int c) {
    constexpr int row = D * (Q8 ? 1 : 2);
    const int x = row == 64 ? (KEY ? 0 : (r >> 1) & 3) : Q8 && KEY ? ((r & 1) << 2) | ((r >> 1) & 3) : r & 7;
    return static_cast<uint32_t>(r * row + ((c ^ x) << 4));
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
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_sum[kWarps];
    __shared__ int s_at;
    __shared__ long long s_before;
    const AttnArgs& a = sp.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int group = warp / R, rw = warp % R;
    const int G = a.q_heads / a.kv_heads;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // The total work, and the request that this CTA's run begins in: each
    // thread sums a stretch of the requests, then one scan over the threads.
    const int per = (a.B + kThreads - 1) / kThreads;
    long long own = 0;
    for (int b = tid * per; b < min((tid + 1) * per, a.B); ++b) own += units(a, request(a, b, 16 * R));
    long long sum = own;
    for (int d = 1; d < 32; d <<= 1) {
        const long long v = __shfl_up_sync(~0u, sum, d);
        if (lane >= d) sum += v;
    }
    if (lane == 31) s_sum[warp] = sum;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) sum += s_sum[w];
        total += s_sum[w];
    }
    const long long ctas = min(static_cast<long long>(gridDim.x), total);
    if (tid == 0) sp.carried[blockIdx.x].last = -1;
    if (blockIdx.x >= ctas) return;
    long long at = blockIdx.x * total / ctas;
    const long long end = (blockIdx.x + 1) * total / ctas;
    if (at >= sum - own && at < sum) {
        long long before = sum - own;
        int b = tid * per;
        for (; b < a.B - 1; ++b) {
            const long long w = units(a, request(a, b, 16 * R));
            if (at < before + w) break;
            before += w;
        }
        s_at = b;
        s_before = before;
    }
    __syncthreads();
    int b = s_at;
    long long before = s_before;  // units of the requests before b

    const uint32_t ring = smem_addr(smem) + group * S::kGroup;
    float2* scales = reinterpret_cast<float2*>(smem + group * S::kGroup + S::kRing);
    const int d_chunks = a.head_dim * S::kElt / 16;

    while (at < end && b < a.B) {
        const Request rq = request(a, b, 16 * R);
        const long long mine = units(a, rq);
        if (at >= before + mine) {
            before += mine;
            ++b;
            continue;
        }
        // The item: head h, row tile rt, tiles [tile0, tile1) of its own; none where the run ends in the fixed units.
        const int weight = rq.tiles + kFixed;
        const int line = static_cast<int>((at - before) / weight);
        const long long item = before + static_cast<long long>(line) * weight;
        const int rt = line % rq.row_tiles, h = line / rq.row_tiles;
        const int tile0 = max(0, static_cast<int>(at - item) - kFixed);
        const int tile1 = static_cast<int>(min(static_cast<long long>(weight), end - item)) - kFixed;
        at = item + weight;
        if (tile1 <= tile0) continue;
        const int rows = rq.n * G, row0 = rt * 16 * R;
        const int low_tile = rq.low / kTile;
        const int tok0 = max(rq.low, (low_tile + tile0) * kTile);
        const int tok1 = min(static_cast<long long>(rq.len), (low_tile + tile1) * static_cast<long long>(kTile));
        const int count = tok1 - tok0 - group * S::kTokens;
        const int stages = count <= 0 ? 0 : (count + S::kGroups * S::kTokens - 1) / (S::kGroups * S::kTokens);

        // ---- loads: lane l knows token l of a stage
        const int* table = a.table + b * a.table_stride;
        auto token_of = [&](int i) { return tok0 + (i * S::kGroups + group) * S::kTokens + (lane & (S::kTokens - 1)); };
        auto page_of = [&](int i) {  // page id of the lane's token, −1 past the end
            const int tok = token_of(i);
            if (i >= stages || tok >= tok1) return -1;
            return __ldg(table + static_cast<int>((static_cast<uint64_t>(tok) * a.page_mul) >> a.page_shift));
        };
        // Scales of a token travel by register for one iteration, then through shared memory.
        float pend_k = 0.f, pend_v = 0.f;
        int pend_at = -1;
        auto put_scales = [&]() {
            if (Q8 && pend_at >= 0 && rw == 0 && lane < S::kTokens)
                scales[pend_at * S::kTokens + lane] = make_float2(pend_k, __log2f(pend_v));
        };
        long long off = -1;     // of the lane's token, in the stage whose keys were asked for last; −1: none
        auto find = [&](int i, int page) {  // stage i
            const int tok = token_of(i);
            const int pi = static_cast<int>((static_cast<uint64_t>(tok) * a.page_mul) >> a.page_shift);
            const int in_page = tok - pi * a.page_size;
            off = -1;
            if (i < stages && tok < tok1) {
                if (page >= 0 && page < a.pages)
                    off = page * a.page_stride + in_page * a.token_stride + h * a.head_stride;
                else
                    record_status(a.status, kStatusInvalid);
            }
            if (Q8) {
                pend_k = pend_v = 0.f;
                if (off >= 0) {
                    const long long s = (static_cast<long long>(page) * a.kv_heads + h) * a.page_size + in_page;
                    pend_k = __bfloat162float(a.k_scales[s]);
                    pend_v = __bfloat162float(a.v_scales[s]);
                }
                pend_at = i < stages ? i % S::kScaleSlots : -1;
            }
        };
        int put = 0;  // ring slot of the next copy
        auto load = [&](bool key, bool any) {  // keys or values of the stage found last
            if (any) {
                const uint32_t dst = ring + put * S::kHalf;
                const uint8_t* src = static_cast<const uint8_t*>(key ? a.k : a.v);
                constexpr int kPerPass = 32 * R / S::kChunks;  // token rows of one pass of the group's lanes
                const int c = (rw * 32 + lane) % S::kChunks, r0 = (rw * 32 + lane) / S::kChunks;
#pragma unroll
                for (int p = 0; p < S::kTokens; p += kPerPass) {
                    const int r = p + r0;
                    const long long o = __shfl_sync(~0u, off, r & 31);
                    const bool there = o >= 0 && c < d_chunks;
                    const uint8_t* from = src + (there ? o * S::kElt + c * 16 : 0);
                    cp_async16_zfill(dst + (key ? place<D, Q8, true>(r, c) : place<D, Q8, false>(r, c)), from, there ? 16 : 0);
                }
            }
            if (++put == S::kSlots) put = 0;
            cp_async_commit();
        };
        // Copy n holds the keys (n even) or values of stage n / 2; copy n + kSlots − 1 is asked for when copy n is
        // there, into the slot of copy n − 1.  asked: the next stage to find.
        int page_next = -1, asked = 0;
        auto load_next = [&](int n) {
            if ((n & 1) == 0) {
                find(asked, page_next);
                ++asked;
                page_next = page_of(asked);
            }
            load((n & 1) == 0, (n >> 1) < stages);
        };
        {
            int first[S::kAhead];
#pragma unroll
            for (int i = 0; i < S::kAhead; ++i) first[i] = page_of(i);
#pragma unroll
            for (int n = 0; n < S::kSlots - 1; ++n) {
                if ((n & 1) == 0) {
                    find(n >> 1, first[n >> 1]);
                    put_scales();
                }
                load((n & 1) == 0, (n >> 1) < stages);
            }
            asked = S::kSlots / 2;
            pend_at = -1;
            page_next = page_of(asked);
        }

        // ---- queries of the thread's rows g and g + 8
        uint32_t q[KS][4];
        int see_lo[2], see_hi[2];   // tokens that a row sees
        float row_scale[2] = {sp.scale_log2, sp.scale_log2};
        {
            const __nv_bfloat16* src[2];
            bool live[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = row0 + rw * 16 + g + 8 * x, j = r / G;
                live[x] = r < rows;
                see_hi[x] = live[x] ? rq.len - rq.n + j + 1 : 0x7fffffff;
                see_lo[x] = live[x] && a.window > 0 ? static_cast<int>(max(0ll, static_cast<long long>(see_hi[x]) - a.window)) : 0;
                src[x] = a.q.data + (live[x] ? (rq.start + j) * a.q.token_stride + (h * G + r % G) * a.q.head_stride : 0);
            }
            if (!Q8) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int k = ks * 16 + 2 * t4 + 8 * (x >> 1);
                        q[ks][x] = live[x & 1] && k < a.head_dim ? *reinterpret_cast<const uint32_t*>(src[x & 1] + k) : 0u;
                    }
            } else {
                // Four values in a row for each k-step and lane, like the keys' codes below; as fp16 after a
                // division of the row by a power of two near its largest value.
                uint2 w[2][KS];
                float most[2] = {0.f, 0.f};
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const int k = (ks >> 2) * 64 + t4 * 16 + (ks & 3) * 4;
                        w[x][ks] = live[x] && k < a.head_dim ? *reinterpret_cast<const uint2*>(src[x] + k) : make_uint2(0, 0);
                        most[x] = fmaxf(most[x], fmaxf(fmaxf(fabsf(bf16_lo(w[x][ks].x)), fabsf(bf16_hi(w[x][ks].x))),
                                                       fmaxf(fabsf(bf16_lo(w[x][ks].y)), fabsf(bf16_hi(w[x][ks].y)))));
                    }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    most[x] = quad_max(most[x]);
                    const int e = min(max(static_cast<int>(__float_as_uint(most[x]) >> 23), 7), 247) - 127;
                    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                    row_scale[x] *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        q[ks][x] = pack_f16(bf16_lo(w[x][ks].x) * down, bf16_hi(w[x][ks].x) * down);
                        q[ks][x + 2] = pack_f16(bf16_lo(w[x][ks].y) * down, bf16_hi(w[x][ks].y) * down);
                    }
                }
            }
        }
        // Tokens before all_hi and from all_lo on are seen by every row of the warp.
        int all_hi, all_lo;
        {
            const int j0 = (row0 + rw * 16) / G, j1 = max(min(row0 + rw * 16 + 15, rows - 1), 0) / G;
            all_hi = rq.len - rq.n + j0 + 1;
            all_lo = a.window > 0 ? static_cast<int>(max(0ll, static_cast<long long>(rq.len) - rq.n + j1 + 1 - a.window)) : 0;
        }

        float o[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i][x] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float mw[2] = {-INFINITY, -INFINITY};  // Q8: largest score + log2(value scale), the weights' reference

        int get = 0;
        for (int i = 0; i < stages; ++i) {
            cp_async_wait<S::kSlots - 2>();
            put_scales();
            group_sync<R>(group);
            pend_at = -1;
            load_next(2 * i + S::kSlots - 1);
            const int base = tok0 + (i * S::kGroups + group) * S::kTokens;
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
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int sub = 0; sub < S::kSub; ++sub) {
                        uint32_t k[4];
                        const int r = sub * 16 + (lane >> 4) * 8 + (lane & 7), c = ks * 2 + ((lane >> 3) & 1);
                        ldmatrix_x4(keys + place<D, Q8, true>(r, c), k);
                        mma16816<false>(s[2 * sub], q[ks], k[0], k[1]);
                        mma16816<false>(s[2 * sub + 1], q[ks], k[2], k[3]);
                    }
            } else {
#pragma unroll
                for (int kb = 0; kb < KS / 4; ++kb)
#pragma unroll
                    for (int y = 0; y < 2 * S::kSub; ++y) {
                        uint4 w = lds128(keys + place<D, Q8, true>(y * 8 + g, kb * 4 + t4));
                        const uint32_t u[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            mma16816<true>(s[y], q[kb * 4 + x], codes_f16(u[x], 0x4140), codes_f16(u[x], 0x4342));
                    }
            }
            float lv[2 * S::kSub][2];  // log2 of the value scales of the lane's tokens
#pragma unroll
            for (int y = 0; y < 2 * S::kSub; ++y) {
                float ks0 = 1.f, ks1 = 1.f;
                if (Q8) {
                    const float4 f = *reinterpret_cast<const float4*>(stage_scales + y * 8 + 2 * t4);
                    ks0 = f.x, lv[y][0] = f.y, ks1 = f.z, lv[y][1] = f.w;
                }
                s[y][0] *= row_scale[0] * ks0;
                s[y][1] *= row_scale[0] * ks1;
                s[y][2] *= row_scale[1] * ks0;
                s[y][3] *= row_scale[1] * ks1;
            }
            // Some row does not see some token of the stage; there are such tokens, too, past the end.
            const bool hidden = min(base + S::kTokens, tok1) > all_hi || base < all_lo;
            const bool partly = hidden || base + S::kTokens > tok1;
            auto sees = [&](int y, int x) {
                const int tok = base + y * 8 + 2 * t4 + (x & 1);
                return tok < min(see_hi[x >> 1], tok1) && tok >= see_lo[x >> 1];
            };
            if (partly) {
#pragma unroll
                for (int y = 0; y < 2 * S::kSub; ++y)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (!sees(y, x)) s[y][x] = -INFINITY;
            }

            // ---- running maximum
            float grown[2] = {m[0], m[1]}, grown_w[2] = {mw[0], mw[1]};
#pragma unroll
            for (int y = 0; y < 2 * S::kSub; ++y)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    grown[x >> 1] = fmaxf(grown[x >> 1], s[y][x]);
                    if (Q8) grown_w[x >> 1] = fmaxf(grown_w[x >> 1], s[y][x] == -INFINITY ? -INFINITY : s[y][x] + lv[y][x & 1]);
                }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                grown[x] = quad_max(grown[x]);
                if (Q8) grown_w[x] = quad_max(grown_w[x]);
            }
            // It grows in the first few stages and seldom after them.
            const bool grew = grown[0] > m[0] || grown[1] > m[1] || (Q8 && (grown_w[0] > mw[0] || grown_w[1] > mw[1]));
            if (__any_sync(~0u, grew)) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float keep_l = m[x] == -INFINITY ? 0.f : ex2(m[x] - grown[x]);
                    const float keep_o = !Q8 ? keep_l : mw[x] == -INFINITY ? 0.f : ex2(mw[x] - grown_w[x]);
                    l[x] *= keep_l;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        o[n][2 * x] *= keep_o;
                        o[n][2 * x + 1] *= keep_o;
                    }
                    m[x] = grown[x];
                    mw[x] = grown_w[x];
                }
            }
            // ---- weights
            const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
            const float refw[2] = {mw[0] == -INFINITY ? 0.f : mw[0], mw[1] == -INFINITY ? 0.f : mw[1]};
#pragma unroll
            for (int y = 0; y < 2 * S::kSub; ++y)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float p = ex2(s[y][x] - ref[x >> 1]);
                    l[x >> 1] += p;
                    s[y][x] = !Q8 ? p : s[y][x] == -INFINITY ? 0.f : ex2(s[y][x] + lv[y][x & 1] - refw[x >> 1]);
                }
            // ---- values
            cp_async_wait<S::kSlots - 2>();
            if (S::kSlots % 2 != 0) put_scales();
            group_sync<R>(group);
            if (S::kSlots % 2 != 0) pend_at = -1;
            load_next(2 * i + S::kSlots);
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
                            // The shuffle's source lane holds the same column's parity, so v is chosen alike there.
                            p[x] = __shfl_sync(~0u, v, from);
                            seen[x] = base + tk < min(see_hi[x], tok1) && base + tk >= see_lo[x];
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint32_t w;
                            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(vals + place<D, Q8, false>(tk, n) + 4 * t4));
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
#pragma unroll
                    for (int n = 0; n < NT / 2; ++n)
#pragma unroll
                        for (int sub = 0; sub < S::kSub; ++sub) {
                            uint32_t v[4];
                            const int r = sub * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), c = n * 2 + (lane >> 4);
                            ldmatrix_x4_trans(vals + place<D, Q8, false>(r, c), v);
                            mma16816<false>(o[2 * n], hi[sub], v[0], v[1]);
                            mma16816<false>(o[2 * n + 1], hi[sub], v[2], v[3]);
                            mma16816<false>(o[2 * n], lo[sub], v[0], v[1]);
                            mma16816<false>(o[2 * n + 1], lo[sub], v[2], v[3]);
                        }
                }
            } else {
                // Weights times value scales, at most 1 by their own reference, as fp16 (2⁻¹¹): an eighth of the
                // result's rounding.
#pragma unroll
                for (int sub = 0; sub < S::kSub; ++sub) {
                    uint32_t p[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        p[x] = pack_f16(s[2 * sub + (x >> 1)][2 * (x & 1)], s[2 * sub + (x >> 1)][2 * (x & 1) + 1]);
                    // Column n of output tile i is value 16·n + i (8·n + i for D = 64) of the row: a lane's
                    // 16 (8) bytes of a token row are its column of 16 (8) tiles.
                    constexpr int kBytes = D == 64 ? 8 : 16;
#pragma unroll
                    for (int hb = 0; hb < NT / kBytes; ++hb) {
                        uint32_t w[4][kBytes / 4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int r = sub * 16 + 2 * t4 + (x & 1) + 8 * (x >> 1);
                            if (kBytes == 16) {
                                const uint4 v = lds128(vals + place<D, Q8, false>(r, hb * 8 + g));
                                w[x][0] = v.x ^ 0x80808080u;
                                w[x][1] = v.y ^ 0x80808080u;
                                w[x][kBytes / 4 - 2] = v.z ^ 0x80808080u;
                                w[x][kBytes / 4 - 1] = v.w ^ 0x80808080u;
                            } else {
                                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                             : "=r"(w[x][0]), "=r"(w[x][1])
                                             : "r"(vals + place<D, Q8, false>(r, g >> 1) + 8 * (g & 1)));
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

        // ---- the groups' sums meet in shared memory: [warp][16 rows][D], then m, mw, l of each row
        __syncthreads();
        float* s_o = reinterpret_cast<float*>(smem);
        float* s_stat = s_o + kWarps * 16 * D;  // [3][warp][16]
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            l[x] = quad_sum(l[x]);
            if (t4 == 0) {
                s_stat[warp * 16 + g + 8 * x] = m[x];
                s_stat[kWarps * 16 + warp * 16 + g + 8 * x] = Q8 ? mw[x] : m[x];
                s_stat[2 * kWarps * 16 + warp * 16 + g + 8 * x] = l[x];
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int col = !Q8 ? n * 8 + 2 * t4 + (x & 1)
                                    : D == 64 ? (2 * t4 + (x & 1)) * 8 + n : (n >> 4) * 128 + (2 * t4 + (x & 1)) * 16 + (n & 15);
                s_o[(warp * 16 + g + 8 * (x >> 1)) * D + col] = o[n][x];
            }
        __syncthreads();
        const bool whole = tile0 == 0 && tile1 == rq.tiles;
        float* part = sp.partial + (2 * static_cast<size_t>(blockIdx.x) + (tile0 > 0 ? 0 : 1)) * partial_floats(R, D);
        for (int x = tid; x < 16 * R * (D / 4); x += kThreads) {
            const int r = x / (D / 4), col = x % (D / 4) * 4, row = row0 + r;
            if (row >= rows || col >= a.head_dim) continue;
            float mm = -INFINITY, mmw = -INFINITY;
#pragma unroll
            for (int k = 0; k < S::kGroups; ++k) {
                mm = fmaxf(mm, s_stat[(k * R * 16) + r]);
                mmw = fmaxf(mmw, s_stat[kWarps * 16 + k * R * 16 + r]);
            }
            const float rm = mm == -INFINITY ? 0.f : mm, rmw = mmw == -INFINITY ? 0.f : mmw;
            float ll = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < S::kGroups; ++k) {
                ll += ex2(s_stat[k * R * 16 + r] - rm) * s_stat[2 * kWarps * 16 + k * R * 16 + r];
                const float f = ex2(s_stat[kWarps * 16 + k * R * 16 + r] - rmw);
                const float4 w = *reinterpret_cast<const float4*>(s_o + (k * R * 16 + r) * D + col);
                v[0] += f * w.x, v[1] += f * w.y, v[2] += f * w.z, v[3] += f * w.w;
            }
            if (whole) {
                const int j = row / G;
                // A row that sees nothing is zeros; one whose scores are all −∞ has no value (0 / 0).
                const float f = rq.len - rq.n + j < 0 ? 0.f : (mmw == -INFINITY ? 0.f : ex2(mmw - mm)) / ll;
                uint2 y = make_uint2(pack_bf16(v[0] * f, v[1] * f), pack_bf16(v[2] * f, v[3] * f));
                *reinterpret_cast<uint2*>(a.out.data + (rq.start + j) * a.out.token_stride +
                                          (h * G + row % G) * a.out.head_stride + col) = y;
            } else {
                if (col == 0) {
                    part[r] = mm;
                    part[16 * R + r] = mmw;
                    part[32 * R + r] = ll;
                }
                *reinterpret_cast<float4*>(part + 48 * R + r * D + col) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
        if (tid == 0 && tile0 == 0 && tile1 < rq.tiles) {
            // The item's last unit is that before the next item; CTA c has the units from ⌊c·total / ctas⌋ on.
            const long long u = at - 1;
            sp.carried[blockIdx.x] = {static_cast<int>(((u + 1) * ctas - 1) / total), h, row0, rows, rq.start, rq.len - rq.n};
        }
        __syncthreads();
    }
}

// Joins the parts of the item that begins in CTA blockIdx.x and ends in a
// later one: its own second part, the later CTAs' first.  A CTA takes one row;
// its warps take the parts in turn, each with a running maximum of its own.
template <int D, int R>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(const __grid_constant__ SplitArgs sp) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Carried c = sp.carried[blockIdx.x];
    const int r = blockIdx.y;
    if (c.last < 0 || c.row0 + r >= c.rows) return;
    const AttnArgs& a = sp.a;
    const int G = a.q_heads / a.kv_heads;
    constexpr int V = D / 32;
    constexpr size_t size = partial_floats(R, D);
    const int parts = c.last - static_cast<int>(blockIdx.x) + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ float s_m[kWarps], s_mw[kWarps], s_l[kWarps], s_v[kWarps][D];
    float mm = -INFINITY, mmw = -INFINITY, ll = 0.f, v[V];
#pragma unroll
    for (int x = 0; x < V; ++x) v[x] = 0.f;
#pragma unroll 4
    for (int k = warp; k < parts; k += kWarps) {
        const float* p = sp.partial + (2 * (static_cast<size_t>(blockIdx.x) + k) + (k == 0)) * size;
        const float pm = p[r], pmw = p[16 * R + r], pl = p[32 * R + r];
        float pv[V];
#pragma unroll
        for (int x = 0; x < V; ++x) pv[x] = lane + 32 * x < a.head_dim ? p[48 * R + r * D + lane + 32 * x] : 0.f;
        const float nm = fmaxf(mm, pm), nw = fmaxf(mmw, pmw);
        const float rm = nm == -INFINITY ? 0.f : nm, rw = nw == -INFINITY ? 0.f : nw;
        ll = ll * ex2(mm - rm) + pl * ex2(pm - rm);
        const float keep = ex2(mmw - rw), f = ex2(pmw - rw);
#pragma unroll
        for (int x = 0; x < V; ++x) v[x] = v[x] * keep + pv[x] * f;
        mm = nm, mmw = nw;
    }
    if (lane == 0) s_m[warp] = mm, s_mw[warp] = mmw, s_l[warp] = ll;
#pragma unroll
    for (int x = 0; x < V; ++x) s_v[warp][lane + 32 * x] = v[x];
    __syncthreads();
    mm = mmw = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w]), mmw = fmaxf(mmw, s_mw[w]);
    const float rm = mm == -INFINITY ? 0.f : mm, rw = mmw == -INFINITY ? 0.f : mmw;
    ll = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) ll += s_l[w] * ex2(s_m[w] - rm);
    const int row = c.row0 + r, j = row / G;
    const float f = c.before + j < 0 ? 0.f : (mmw == -INFINITY ? 0.f : ex2(mmw - mm)) / ll;
    __nv_bfloat16* out = a.out.data + (c.start + j) * a.out.token_stride + (c.head * G + row % G) * a.out.head_stride;
    for (int col = threadIdx.x; col < a.head_dim; col += kThreads) {
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) y += s_v[w][col] * ex2(s_mw[w] - rw);
        out[col] = __float2bfloat16_rn(y * f);
    }
}

int dim_of(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

// Warps (of 16 rows) that share a stage: what the requests' rows need on the
// average, at most 4.
int row_warps(int32_t B, int64_t T, int G) {
    const int64_t rows = (T + B - 1) / B * G;
    return rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
}

template <int D, bool Q8, int R>
cudaError_t run(SplitArgs sp, void* workspace, const DeviceInfo& dev, cudaStream_t stream) {
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
    const int grid = std::min(per_sm * dev.sm_count, kMaxCtas);
    sp.carried = static_cast<Carried*>(workspace);
    sp.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kMaxCtas * 32);
    attn_split_kernel<D, Q8, R><<<grid, kThreads, S::kSmem, stream>>>(sp);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 16 * R);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<D, R>, sp);
}

template <int D, bool Q8>
cudaError_t run_rows(const SplitArgs& sp, void* workspace, const DeviceInfo& dev, cudaStream_t stream) {
    const int R = row_warps(sp.a.B, sp.a.T, sp.a.q_heads / sp.a.kv_heads);
    if (R == 1) return run<D, Q8, 1>(sp, workspace, dev, stream);
    if (R == 2) return run<D, Q8, 2>(sp, workspace, dev, stream);
    return run<D, Q8, 4>(sp, workspace, dev, stream);
}

template <bool Q8>
cudaError_t run_dim(const SplitArgs& sp, void* workspace, const DeviceInfo& dev, cudaStream_t stream) {
    const int D = dim_of(sp.a.head_dim);
    if (D == 64) return run_rows<64, Q8>(sp, workspace, dev, stream);
    if (D == 128) return run_rows<128, Q8>(sp, workspace, dev, stream);
    return run_rows<256, Q8>(sp, workspace, dev, stream);
}

}  // namespace

size_t attn_decode_workspace_bytes(int32_t B, int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    static_assert(sizeof(Carried) <= 32, "a CTA's record fits its place in the workspace");
    const int R = B > 0 ? row_warps(B, T, q_heads / kv_heads) : 1;
    return kMaxCtas * 32 + 2 * kMaxCtas * partial_floats(R, dim_of(head_dim)) * sizeof(float);
}

cudaError_t launch_attn_decode(AttnArgs a, bool q8, void* workspace, const DeviceInfo& dev, cudaStream_t stream) {
    divide_by(a.page_size, &a.page_mul, &a.page_shift);
    SplitArgs sp = {};
    sp.a = a;
    sp.scale_log2 = a.scale * 1.4426950408889634f;
    return q8 ? run_dim<true>(sp, workspace, dev, stream) : run_dim<false>(sp, workspace, dev, stream);
}

}  // namespace w4
