// Attention over the paged cache where many rows read each key-value head
// (verify passes of several drafts): tcgen05 products, one CTA to an SM.
//
// The pass is that of the kernel for few rows: o = Σ_t 2^(s_t − m) v_t /
// Σ_t 2^(s_t − m) in one pass over the tokens, the work in equal pieces, parts
// of shared items joined by the CTA that finishes last.  What differs is what
// bounds it: with R rows a byte of keys and values takes 2·R operations, and
// the m16n8k16 MMAs of the other kernel reach a quarter of the tensor cores'
// rate (104 rows of 128 over 16 requests of 1024 to 8192 tokens: 255 µs with
// 16 rows to a pass, 196 with 64; here 71, of which the cache's bytes are 39).
//
//   S [128 rows, TT tokens] = Q [rows, D] · Kᵀ     both from shared memory
//   O [128 rows, D]        += P [rows, tokens] · V  P from tensor memory
//
// A tile is TT = 128 tokens (64 at D = 256: 64 KB of keys and values either
// way).  Warps 0 to 3 hold a row per thread: they read S from tensor memory,
// twice (the largest score, then the weights), so that a row's statistics need
// no exchange between threads, and write the weights over it, as two bf16 each
// (one alone would err as much as the result's rounding).  That takes them
// about 3000 cycles a tile of 128 tokens, as long as its bytes take at D = 128.
// The next warps copy the tokens' rows by cp.async, from pages of any size, into
// a ring of slots, keys and values in turn.  The last warp issues the products:
// the scores of tile i + 1 while the weights of tile i are made.
// Tensor memory: S of three tiles from column 0, then O.
//
// Format 8: codes are exact as bf16, so the products are those of format 16,
// with the key scales applied to the scores and the value scales to the
// weights.  Codes arrive in slots of their own and eight warps turn them to
// bf16 (96 µs for the call above, 99 with four; 787 and 875 for 32 rows over 64
// requests of 8192 to 16384).  Bound by the row threads' and these warps'
// instructions, the bytes being half of format 16's.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "w4_attn_common.cuh"
#include "w4_attn_tc.cuh"
#include "w4_attn_tc.h"
#include "w4_device.cuh"
#include "w4_kv.h"
#include "w4_tcgen05.cuh"

namespace w4 {
namespace {

constexpr int kRows = 128;
constexpr int kSoftmaxWarps = 4;
constexpr int kFixed = 2;  // an item's fixed cost in tiles
constexpr uint32_t kTmemCols = 512;

template <int D, bool Q8>
struct Shape {
    static constexpr int kLoadWarps = Q8 ? 8 : 4, kMmaWarp = kSoftmaxWarps + kLoadWarps, kThreads = 32 * (kMmaWarp + 1);
    static constexpr int kTile = D == 256 ? 64 : 128;
    static constexpr uint32_t kColO = D == 256 ? 256 : 384;
    static constexpr int kBlocks = D / 64;            // 128-byte columns of a row
    static constexpr int kSlot = kTile * D * 2;       // keys or values of a tile
    static constexpr int kSlots = Q8 ? (D == 256 ? 3 : 4) : D == 256 ? 4 : 6;  // what shared memory holds
    static constexpr int kQ = kRows * D * 2;
    // Format 8: tiles of codes on their way, in slots of their own.
    static constexpr int kAhead = 2, kRaw = kTile * D, kRawSlots = Q8 ? kAhead + 1 : 0;
    // At least what keeps a second CTA, which would wait for tensor memory, off the SM.
    static constexpr int kNeed = 1024 + kQ + kSlots * kSlot + kRawSlots * kRaw;
    static constexpr int kSmem = kNeed > 120 * 1024 ? kNeed : 120 * 1024;
};

__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxWarps * 32) : "memory"); }

template <int D, bool Q8, class SP>
__global__ void __launch_bounds__(Shape<D, Q8>::kThreads, 1) attn_tc_kernel(const __grid_constant__ SP sp) {
    using S = Shape<D, Q8>;
    constexpr int TT = S::kTile, NS = S::kSlots, kLoadWarps = S::kLoadWarps, kMmaWarp = S::kMmaWarp;
    extern __shared__ uint8_t smem_raw[];
    // s_values: the products of even and of odd tiles are in O; apart, since a wait may look two tiles back.
    __shared__ __align__(8) uint64_t s_full[NS], s_empty[NS], s_scores[3], s_weights[3], s_values[2], s_queries;
    // Format 8, by the tile's score buffer: the tokens' key scales (times that of the scores) and value scales.
    __shared__ __align__(8) uint64_t s_scaled[3];
    __shared__ __align__(16) float s_scale[Q8 ? 3 : 1][2][Q8 ? TT : 4];
    __shared__ uint32_t s_tmem;
    __shared__ bool s_last;
    const AttnArgs& a = sp.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t q_smem = (smem_addr(smem_raw) + 1023) & ~1023u, ring = q_smem + S::kQ;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_addr(&s_full[i]), kLoadWarps * 32);
            mbar_init(smem_addr(&s_empty[i]), 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(smem_addr(&s_scores[i]), 1);
            mbar_init(smem_addr(&s_weights[i]), kSoftmaxWarps * 32);
            mbar_init(smem_addr(&s_scaled[i]), kLoadWarps * 32);
        }
        mbar_init(smem_addr(&s_values[0]), 1);
        mbar_init(smem_addr(&s_values[1]), 1);
        mbar_init(smem_addr(&s_queries), kSoftmaxWarps * 32);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    let_next_start(sp);
    Walk<TT, kRows, kFixed> walk;
    if (!walk.template find<S::kThreads>(sp)) {
        end_after_the_one_before(sp);
        return;
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&s_tmem), kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool alive = true;

    if (warp == kMmaWarp) {
        // ------------------------------------------------------ products
        // A factor below zero turns the queries' signs over.
        const uint32_t qk_idesc = idesc_bf16(TT) | (sp.flip ? 1u << 13 : 0u), pv_idesc = idesc_bf16(D) | 1u << 16;  // B (values) N-major
        Turn slot;            // of the next tile's keys or values, as they come
        Turn next, now;       // score buffers of the tile to be scored next and of the one whose values are next
        uint32_t tile = 0, items = 0;
        for (Item it; walk.next(sp, it);) {
            const int tiles = tiles_of<TT>(it);
            if (tiles == 0) continue;
            wait_or_report(smem_addr(&s_queries), items++ & 1, alive, a.status);
            auto scores = [&]() {  // of the tile whose keys come next
                wait_or_report(smem_addr(&s_full[slot.place]), slot.round, alive, a.status);
                fence_async_smem();  // the copies were made through the generic proxy
                tc_fence_after();
                const uint32_t keys = ring + slot.place * S::kSlot;
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_bf16(tmem + next.place * TT, sw128_desc(q_smem + (ks >> 2) * kRows * 128 + (ks & 3) * 32),
                                 sw128_desc(keys + (ks >> 2) * TT * 128 + (ks & 3) * 32), qk_idesc, ks > 0);
                    mma_commit(smem_addr(&s_empty[slot.place]));
                    mma_commit(smem_addr(&s_scores[next.place]));
                }
                __syncwarp();
                slot.step(NS);
                next.step(3);
            };
            scores();
            for (int i = 0; i < tiles; ++i, ++tile) {
                // The tile's values lie after its keys; the next tile's keys after those.
                const Turn values = slot;
                slot.step(NS);
                if (i + 1 < tiles) {
                    // Its scores go where the weights of tile − 2 are, which must have been used.
                    if (i > 1) wait_or_report(smem_addr(&s_values[tile & 1]), (tile - 2) >> 1 & 1, alive, a.status);
                    scores();
                }
                wait_or_report(smem_addr(&s_full[values.place]), values.round, alive, a.status);
                wait_or_report(smem_addr(&s_weights[now.place]), now.round, alive, a.status);
                fence_async_smem();
                tc_fence_after();
                const uint32_t vals = ring + values.place * S::kSlot, weights = tmem + now.place * TT;
                if (elect_one()) {
                    // Sixteen tokens' weights: 8 columns of their upper halves, 16 columns further the lower ones.
#pragma unroll
                    for (int ks = 0; ks < TT / 16; ++ks) {
                        const uint64_t desc = values_desc(vals + ks * 2048, TT * 128);
                        mma_bf16_tmem_a(tmem + S::kColO, weights + (ks >> 1) * 32 + (ks & 1) * 8, desc, pv_idesc, 1);
                        mma_bf16_tmem_a(tmem + S::kColO, weights + (ks >> 1) * 32 + (ks & 1) * 8 + 16, desc, pv_idesc, 1);
                    }
                    mma_commit(smem_addr(&s_empty[values.place]));
                    mma_commit(smem_addr(&s_values[tile & 1]));
                }
                __syncwarp();
                now.step(3);
            }
        }
    } else if (warp >= kSoftmaxWarps) {
        // -------------------------------------------------------- copies
        // A warp copies TT / 4 tokens of each tile; lane l knows token l of them.
        // Format 8: into slots of codes, which the lane that copied them turns to bf16, kAhead half tiles later.
        constexpr int kMine = TT / kLoadWarps, kSub = Q8 ? 1 : kMine / 16, kChunks = D * (Q8 ? 1 : 2) / 16;
        constexpr int kPerPass = 32 / kChunks;  // token rows of one pass of the warp's lanes (D ≤ 256)
        const int my_row = (warp - kSoftmaxWarps) * kMine, d_chunks = a.head_dim * (Q8 ? 1 : 2) / 16;
        const int load_c = lane % kChunks, load_r = lane / kChunks;
        Turn slot;
        slot.round = 1;  // the ring's first round finds its slots free
        // Format 8.  The scales of the lane's token travel by register until its codes are there.  A tile's go where
        // those of the third tile before were: its values' slot has been filled anew, so they have been used.
        struct Scales {
            __nv_bfloat16 k, v;
        };
        const Scales none = {__ushort_as_bfloat16(0), __ushort_as_bfloat16(0)};
        Scales found = none, older = none;
        Turn scaled;
        const uint32_t raw = ring + NS * S::kSlot + ((warp - kSoftmaxWarps) * kMine * kChunks + lane) * 16;
        int asked = 0, raw_ask = 0, raw_take = 0;
        // Asks for half a tile of codes (or, past the last, for nothing) and turns that of kAhead before.
        auto half_tile = [&](bool key, bool any, long long off) {
            if (any) {
                const uint8_t* src = static_cast<const uint8_t*>(key ? a.k : a.v) + load_c * 16;
#pragma unroll
                for (int p = 0; p < kMine; p += kPerPass) {
                    const long long o = __shfl_sync(~0u, off, p + load_r);
                    const bool there = o >= 0 && load_c < d_chunks;
                    cp_async16_zfill(raw + raw_ask * S::kRaw + p * kChunks * 16, there ? src + o : static_cast<const uint8_t*>(a.k), there ? 16 : 0);
                }
            }
            cp_async_commit();
            if (++raw_ask == S::kAhead + 1) raw_ask = 0;
            if (asked < S::kAhead) {
                ++asked;
                return;
            }
            cp_async_wait<S::kAhead>();
            wait_or_report(smem_addr(&s_empty[slot.place]), slot.round, alive, a.status);
            const bool keys = S::kAhead % 2 == 0 ? key : !key;
            const uint32_t dst = ring + slot.place * S::kSlot;
            // A 16-byte chunk of codes makes two of values; lanes in the upper half of 128 bytes of codes write the second
            // one first, so that eight lanes' chunks fall in different banks.
            const int second = D > 64 && (load_c & 4) ? 1 : 0;
#pragma unroll 4
            for (int p = 0; p < kMine; p += kPerPass) {
                const uint4 w = lds128(raw + raw_take * S::kRaw + p * kChunks * 16);
                const uint2 x = codes_bf16(w.x), y = codes_bf16(w.y), z = codes_bf16(w.z), u = codes_bf16(w.w);
                const uint4 lo = make_uint4(x.x, x.y, y.x, y.y), hi = make_uint4(z.x, z.y, u.x, u.y);
                sts128(dst + place<TT>(my_row + p + load_r, 2 * load_c + second), second ? hi : lo);
                sts128(dst + place<TT>(my_row + p + load_r, 2 * load_c + (second ^ 1)), second ? lo : hi);
            }
            if (++raw_take == S::kAhead + 1) raw_take = 0;
            if (keys) {
                if (lane < kMine) {
                    s_scale[scaled.place][0][my_row + lane] = __bfloat162float(older.k) * sp.scale_log2;
                    s_scale[scaled.place][1][my_row + lane] = __bfloat162float(older.v);
                }
                mbar_arrive(smem_addr(&s_scaled[scaled.place]));
                scaled.step(3);
            }
            mbar_arrive(smem_addr(&s_full[slot.place]));
            slot.step(NS);
        };
        for (Item it; walk.next(sp, it);) {
            const int base0 = it.tok0 & ~15, tiles = tiles_of<TT>(it);
            const int* table = a.table + it.b * a.table_stride;
            auto page_of = [&](int i) {  // page id of the lane's token, −1 outside the piece
                const int tok = base0 + i * TT + my_row + (lane & (kMine - 1));
                return i < tiles && tok >= it.tok0 && tok < it.tok1 ? __ldg(table + sp.page_index(tok)) : -1;
            };
            int page_next = page_of(0);
            for (int i = 0; i < tiles; ++i) {
                const int tok = base0 + i * TT + my_row + (lane & (kMine - 1)), page = page_next;
                page_next = page_of(i + 1);
                long long off = -1;
                if (tok >= it.tok0 && tok < it.tok1) {
                    if (page >= 0 && page < a.pages)
                        off = page * a.page_stride + (tok - sp.page_index(tok) * a.page_size) * a.token_stride + it.h * a.head_stride;
                    else
                        record_status(a.status, kStatusInvalid);
                }
                if constexpr (Q8) {
                    older = found;
                    found = none;
                    if (off >= 0) {
                        const long long at = (static_cast<long long>(page) * a.kv_heads + it.h) * a.page_size + (tok - sp.page_index(tok) * a.page_size);
                        found.k = a.k_scales[at];
                        found.v = a.v_scales[at];
                    }
                    half_tile(true, true, off);
                    half_tile(false, true, off);
                } else {
                    long long off0[kSub];  // of the first token of each 16
#pragma unroll
                    for (int sub = 0; sub < kSub; ++sub) off0[sub] = __shfl_sync(~0u, off, 16 * sub);
                    const long long mine = kSub == 2 && (lane & 16) ? off0[kSub - 1] : off0[0];
                    const bool even = __all_sync(~0u, mine >= 0 && off == mine + (lane & 15) * a.token_stride) && d_chunks == kChunks;
#pragma unroll
                    for (int key = 1; key >= 0; --key) {
                        wait_or_report(smem_addr(&s_empty[slot.place]), slot.round, alive, a.status);
                        const uint32_t dst = ring + slot.place * S::kSlot;
                        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(key ? a.k : a.v);
                        if (even) {
#pragma unroll
                            for (int sub = 0; sub < kSub; ++sub) {
                                const __nv_bfloat16* from = src + off0[sub] + load_r * a.token_stride + load_c * 8;
#pragma unroll
                                for (int p = 0; p < 16; p += kPerPass) {
                                    cp_async16(dst + place<TT>(my_row + sub * 16 + p + load_r, load_c), from);
                                    from += kPerPass * a.token_stride;
                                }
                            }
                        } else {
#pragma unroll 4
                            for (int p = 0; p < kMine; p += kPerPass) {
                                const long long o = __shfl_sync(~0u, off, p + load_r);
                                const bool there = o >= 0 && load_c < d_chunks;
                                cp_async16_zfill(dst + place<TT>(my_row + p + load_r, load_c), src + (there ? o + load_c * 8 : 0), there ? 16 : 0);
                            }
                        }
                        cp_async_arrive(smem_addr(&s_full[slot.place]));
                        slot.step(NS);
                    }
                }
            }
        }
        if constexpr (Q8) {
            if (asked > 0) {
                older = found;
#pragma unroll 1
                for (int i = 0; i < S::kAhead; ++i) half_tile(i % 2 == 0, false, 0);
            }
        }
        cp_async_wait_all();
    } else {
        // ------------------------------------------- a row in every thread
        const uint32_t mine = tmem + (static_cast<uint32_t>(warp * 32) << 16);  // the warp's lanes
        Turn slot;  // of the tile's values
        slot.step(NS);
        uint32_t tile = 0;
        Turn now;  // of the tile's scores
        // The queries of an item are asked for before the sums of the one before it go out: a row by D / 8 lanes.  Not those
        // of an item without tokens: nothing reads or waits for them, and the next item's copies to the same places would
        // be under way together with them, in no order.
        auto ask = [&](const Item& n) {
            if (tiles_of<TT>(n) == 0) return;
            constexpr int kChunks = D / 8, kPerPass = kSoftmaxWarps * 32 / kChunks;
            const int c = tid % kChunks;
#pragma unroll 4
            for (int p = 0; p < kRows; p += kPerPass) {
                const int r = p + tid / kChunks, row = n.row0 + r, jr = sp.over_G(row);
                const bool there = row < n.rows && 8 * c < a.head_dim;
                const __nv_bfloat16* src = a.q.data + (there ? (n.start + jr) * a.q.token_stride + (n.h * sp.G + row - jr * sp.G) * a.q.head_stride + 8 * c : 0);
                cp_async16_zfill(q_smem + place<kRows>(r, c), src, there ? 16 : 0);
            }
        };
        Item it;
        bool more = walk.next(sp, it);
        if (more) ask(it);
        while (more) {
            const int base0 = it.tok0 & ~15, tiles = tiles_of<TT>(it);
            const int row = it.row0 + tid, j = sp.over_G(row);
            const bool live = row < it.rows;
            const int see_hi = live ? it.before + j + 1 : 0x7fffffff;  // tokens that the row sees
            const int see_lo = live && a.window > 0 ? static_cast<int>(max(0ll, static_cast<long long>(see_hi) - a.window)) : 0;
            // Tokens before all_hi and from all_lo on are seen by every row of the item.
            const int all_hi = it.before + sp.over_G(it.row0) + 1;
            const int all_lo = a.window > 0 ? static_cast<int>(max(0ll, static_cast<long long>(it.before) +
                                                                          sp.over_G(min(it.row0 + kRows, it.rows) - 1) + 1 - a.window)) : 0;
            if (tiles > 0) {
                cp_async_wait_all();
                fence_async_smem();
                uint32_t zero[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) zero[x] = 0;
#pragma unroll
                for (int c = 0; c < D; c += 32) tmem_st32(mine + S::kColO + c, zero);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_addr(&s_queries));
            }
            float m = -INFINITY, l = 0.f;  // reference score, unscaled (format 8: to base 2); sum of the weights
            const float unit = Q8 ? 1.f : sp.scale_log2;
            for (int i = 0; i < tiles; ++i, ++tile, now.step(3), slot.step(NS), slot.step(NS)) {
                const int base = base0 + i * TT;
                const bool hidden = min(base + TT, it.tok1) > all_hi || max(base, it.tok0) < all_lo;
                const bool partly = hidden || base + TT > it.tok1 || base < it.tok0;
                // Columns that the row sees: from lo on, `wide` of them.
                const int lo = max(see_lo, it.tok0) - base, wide = max(min(see_hi, it.tok1) - base - lo, 0);
                auto sees = [&](int column) { return static_cast<unsigned>(column - lo) < static_cast<unsigned>(wide); };
                const uint32_t scores = mine + now.place * TT;
                wait_or_report(smem_addr(&s_scores[now.place]), now.round, alive, a.status);
                tc_fence_after();
                const float(*const scale)[Q8 ? TT : 4] = s_scale[Q8 ? now.place : 0];
                // v times the key scales from column c on
                auto scale_scores = [&](uint32_t(&v)[32], int c) {
                    if (Q8)
#pragma unroll
                        for (int x = 0; x < 32; x += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(&scale[0][c + x]);
                            v[x] = __float_as_uint(__uint_as_float(v[x]) * f.x);
                            v[x + 1] = __float_as_uint(__uint_as_float(v[x + 1]) * f.y);
                            v[x + 2] = __float_as_uint(__uint_as_float(v[x + 2]) * f.z);
                            v[x + 3] = __float_as_uint(__uint_as_float(v[x + 3]) * f.w);
                        }
                };
                if (Q8) wait_or_report(smem_addr(&s_scaled[now.place]), now.round, alive, a.status);
                // ---- reference
                float grown = m;
                auto largest = [&](auto some) {  // of the scores that the row sees: all of the tile's, or some
#pragma unroll 1
                    for (int c = 0; c < TT; c += 32) {
                        uint32_t v[32];
                        tmem_ld32(scores + c, v);
                        scale_scores(v, c);
#pragma unroll
                        for (int x = 0; x < 32; ++x) {
                            const float f = __uint_as_float(v[x]);
                            grown = fmaxf(grown, !decltype(some)::value || sees(c + x) ? f : -INFINITY);
                        }
                    }
                };
                if (partly)
                    largest(std::true_type());
                else
                    largest(std::false_type());
                auto values_so_far = [&]() {  // the products before this tile's are in O
                    if (i > 0) wait_or_report(smem_addr(&s_values[(tile - 1) & 1]), (tile - 1) >> 1 & 1, alive, a.status);
                    tc_fence_after();
                };
                const float by = (grown - m) * unit;
                if (__any_sync(~0u, by > 8.f)) {
                    const float keep = m == -INFINITY ? 0.f : ex2(-by);
                    if (i > 0) {
                        values_so_far();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t v[32];
                            tmem_ld32(mine + S::kColO + c, v);
#pragma unroll
                            for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * keep);
                            tmem_st32(mine + S::kColO + c, v);
                        }
                        tmem_wait_st();
                    }
                    l *= keep;
                    m = grown;
                }
                const float ref = m == -INFINITY ? 0.f : m * unit;

                // ---- values that are not finite, of tokens that some rows do not see: 0 · ∞ would spoil those rows.
                // They are made 0 for the product and added here to the rows that see them.
                if (!Q8 && hidden) {
                    const uint32_t vals = ring + slot.place * S::kSlot;
                    wait_or_report(smem_addr(&s_full[slot.place]), slot.round, alive, a.status);
                    bool odd = false;
                    for (int x = tid; x < TT * S::kBlocks * 8; x += kSoftmaxWarps * 32) {
                        const uint4 w = lds128(vals + x * 16);
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) odd |= (u[y] & 0x7F80u) == 0x7F80u || (u[y] & 0x7F800000u) == 0x7F800000u;
                    }
                    if (tid == 0) s_last = false;
                    rows_sync();
                    if (odd) s_last = true;
                    rows_sync();
                    if (s_last) {
                        values_so_far();
#pragma unroll 1
                        for (int tk = 0; tk < TT; ++tk) {
                            bool bad = false;  // the token's row has such a value: the same for all threads
                            for (int c = 0; c < D / 8; ++c) {
                                const uint4 w = lds128(vals + place<TT>(tk, c));
                                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                for (int y = 0; y < 4; ++y) bad |= (u[y] & 0x7F80u) == 0x7F80u || (u[y] & 0x7F800000u) == 0x7F800000u;
                            }
                            if (!bad) continue;
                            uint32_t sv[32];
                            tmem_ld32(scores + (tk & ~31), sv);
                            float score = 0.f;
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if (x == (tk & 31)) score = __uint_as_float(sv[x]);
                            const bool seen = sees(tk);
                            const float p = seen ? ex2(fmaf(score, sp.scale_log2, -ref)) : 0.f;
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t v[32];
                                tmem_ld32(mine + S::kColO + c, v);
#pragma unroll
                                for (int x = 0; x < 32; x += 8) {
                                    const uint4 w = lds128(vals + place<TT>(tk, (c + x) / 8));
                                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                    for (int y = 0; y < 8; ++y) {
                                        const float value = y & 1 ? bf16_hi(u[y >> 1]) : bf16_lo(u[y >> 1]);
                                        if (seen) v[x + y] = __float_as_uint(__uint_as_float(v[x + y]) + p * value);
                                    }
                                }
                                tmem_st32(mine + S::kColO + c, v);
                            }
                            tmem_wait_st();
                            rows_sync();  // every row has read the token's values
                            for (int c = tid; c < D / 8; c += kSoftmaxWarps * 32) sts128(vals + place<TT>(tk, c), make_uint4(0, 0, 0, 0));
                        }
                        fence_async_smem();
                    }
                }
                // ---- weights, over the scores: of 32 tokens the upper halves in 16 columns, then the lower ones
                float sums[4] = {l, 0.f, 0.f, 0.f};
                auto weights = [&](auto some) {
#pragma unroll 1
                    for (int c = 0; c < TT; c += 32) {
                        uint32_t v[32], w[32];
                        tmem_ld32(scores + c, v);
                        scale_scores(v, c);
#pragma unroll
                        for (int x = 0; x < 32; x += 2) {
                            float s0 = __uint_as_float(v[x]), s1 = __uint_as_float(v[x + 1]);
                            const bool see0 = !decltype(some)::value || sees(c + x), see1 = !decltype(some)::value || sees(c + x + 1);
                            s0 = see0 ? s0 : -INFINITY;
                            s1 = see1 ? s1 : -INFINITY;
                            float p0 = ex2(Q8 ? s0 - ref : fmaf(s0, unit, -ref)), p1 = ex2(Q8 ? s1 - ref : fmaf(s1, unit, -ref));
                            sums[x & 2] += p0;
                            sums[(x & 2) + 1] += p1;
                            if (Q8) {  // (a hidden token's scale may be anything)
                                const float2 f = *reinterpret_cast<const float2*>(&scale[1][c + x]);
                                p0 = see0 ? p0 * f.x : 0.f;
                                p1 = see1 ? p1 * f.y : 0.f;
                            }
                            // Both halves cut off, not rounded (roundings to bf16 would share the exponentials' slow
                            // pipe): the lower ones take what the upper ones leave, to 16 bits in all, at most 2⁻¹⁵ and
                            // on the average 2⁻¹⁷ of the weight too low.
                            const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
                            w[x >> 1] = __byte_perm(u0, u1, 0x7632);
                            w[16 + (x >> 1)] = __byte_perm(__float_as_uint(p0 - __uint_as_float(u0 & 0xFFFF0000u)),
                                                           __float_as_uint(p1 - __uint_as_float(u1 & 0xFFFF0000u)), 0x7632);
                        }
                        tmem_st32(scores + c, w);
                    }
                };
                if (partly)
                    weights(std::true_type());
                else
                    weights(std::false_type());
                l = (sums[0] + sums[1]) + (sums[2] + sums[3]);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_addr(&s_weights[now.place]));
            }
            // ---- the row's sums
            Item after;
            more = walk.next(sp, after);
            if (more) ask(after);
            if (tiles > 0) wait_or_report(smem_addr(&s_values[(tile - 1) & 1]), (tile - 1) >> 1 & 1, alive, a.status);
            tc_fence_after();
            const bool whole = it.whole(), none = it.before + j < 0;
            const Parts<kRows, D> parts(sp, walk, it, kFixed);
            const int k_own = static_cast<int>(blockIdx.x) - parts.first;
            float* const part = parts.at(k_own);
            // For the join, row by row.  (Up to 128 values a head, prefixes have a kernel of their own.)
            const bool leave = D > 128 && sp.pass() == kPrefixes && !whole;
            if (leave && live) {
                reinterpret_cast<float2*>(part)[tid] = make_float2(m * unit, fminf(l, 3e38f));
                if (k_own == 0)
                    a.sums[static_cast<size_t>(it.start + j) * a.q_heads + it.h * sp.G + row - j * sp.G] =
                        make_float4(0.f, 0.f, __int_as_float(parts.count), __int_as_float(parts.first << 8 | tid));
            } else if (!whole && live) {
                part[tid] = m * unit;
                part[kRows + tid] = fminf(l, 3e38f);
            }
            // A row that sees nothing is zeros; one whose scores are all −∞ has no value (0 · 1 / 0).
            __nv_bfloat16* const to = a.out.data + (live ? (it.start + j) * a.out.token_stride + (it.h * sp.G + row - j * sp.G) * a.out.head_stride : 0);
            // 32 of the row's values from column c on, weights of reference top with the sum `total`
            auto put = [&](int c, const uint32_t (&v)[32], float top, float total) {
                if (sp.pass() != kAlone) {
                    const size_t at = static_cast<size_t>(it.start + j) * a.q_heads + it.h * sp.G + row - j * sp.G;
                    if (c == 0) a.sums[at] = row_sums(sp, it, none, top, total);
#pragma unroll
                    for (int x = 0; x < 32; x += 4)
                        if (c + x < a.head_dim) *reinterpret_cast<uint4*>(a.sum_values + at * a.head_dim + c + x) = make_uint4(v[x], v[x + 1], v[x + 2], v[x + 3]);
                    return;
                }
                const float f = 1.f / total;
#pragma unroll
                for (int x = 0; x < 32; x += 8) {
                    uint32_t y[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        y[z] = none ? 0u : pack_bf16(__uint_as_float(v[x + 2 * z]) * f, __uint_as_float(v[x + 2 * z + 1]) * f);
                    if (c + x < a.head_dim) *reinterpret_cast<uint4*>(to + c + x) = make_uint4(y[0], y[1], y[2], y[3]);
                }
            };
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t v[32];
                tmem_ld32(mine + S::kColO + c, v);
                if (live && leave) {
#pragma unroll
                    for (int x = 0; x < 32; x += 4) *reinterpret_cast<uint4*>(part + 2 * kRows + tid * D + c + x) = make_uint4(v[x], v[x + 1], v[x + 2], v[x + 3]);
                } else if (live && !whole) {
#pragma unroll
                    for (int x = 0; x < 32; ++x) part[(2 + c + x) * kRows + tid] = __uint_as_float(v[x]);
                } else if (live) {
                    put(c, v, m * unit, l);
                }
                __syncwarp();
            }
            tc_fence_before();
            rows_sync();
            // Parts as [reference, sum, D columns][row], so that neighbouring threads' rows lie side by side.
            if (!whole && !leave)
                parts.finish(sp, s_last, rows_sync, [&](int k0, int n, int step, bool last) {
                    // This CTA's own part is still in tensor memory (the item's, when it is a group's that is joined).
                    const int own = step == 1 ? static_cast<int>(blockIdx.x) - parts.first - k0 : -1;
                    auto at = [&](int k) { return parts.at(k0 + min(k, n - 1) * step) + tid; };
                    float mm = -INFINITY, ll = 0.f;
#pragma unroll 4
                    for (int k = 0; k < n; ++k) mm = fmaxf(mm, live ? __ldcg(at(k)) : 0.f);
                    const float rm = mm == -INFINITY ? 0.f : mm;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t v[32];
                        float sum = 0.f;
#pragma unroll
                        for (int x = 0; x < 32; ++x) v[x] = 0;
                        auto fetch = [&](int k, uint32_t (&u)[32]) {
                            const float* p = at(k) + (2 + c) * kRows;
                            if (k == own) {
                                tmem_ld32(mine + S::kColO + c, u);
                            } else {
#pragma unroll
                                for (int x = 0; x < 32; ++x) u[x] = __float_as_uint(__ldcg(p + x * kRows));
                            }
                        };
                        auto add = [&](int k, const uint32_t (&u)[32]) {
                            if (k >= n || !live) return;
                            const float f = ex2(__ldcg(at(k)) - rm);
                            sum += f * __ldcg(at(k) + kRows);
#pragma unroll
                            for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(fmaf(f, __uint_as_float(u[x]), __uint_as_float(v[x])));
                        };
#pragma unroll 1
                        for (int k = 0; k < n; k += 2) {  // two parts' loads in flight
                            uint32_t u0[32], u1[32];
                            fetch(k, u0);
                            fetch(k + 1, u1);
                            add(k, u0);
                            add(k + 1, u1);
                        }
                        ll = sum;
                        if (live && last) put(c, v, mm, ll);
                        if (live && !last)
#pragma unroll
                            for (int x = 0; x < 32; ++x) parts.at(k0)[(2 + c + x) * kRows + tid] = __uint_as_float(v[x]);
                    }
                    if (live && !last) {
                        parts.at(k0)[tid] = mm;
                        parts.at(k0)[kRows + tid] = fminf(ll, 3e38f);
                    }
                });
            it = after;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    end_after_the_one_before(sp);
}

template <int D, bool Q8, class SP>
cudaError_t run(const SP& sp, int grid, cudaStream_t stream) {
    using S = Shape<D, Q8>;
    static std::atomic<bool> ready[kMaxDevices];  // the kernel may use its shared memory on this device
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err != cudaSuccess) return err;
    if (!ready[device & (kMaxDevices - 1)].load(std::memory_order_relaxed)) {
        err = cudaFuncSetAttribute(attn_tc_kernel<D, Q8, SP>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (err != cudaSuccess) return err;
        ready[device & (kMaxDevices - 1)].store(true, std::memory_order_relaxed);
    }
    return launch_pass(attn_tc_kernel<D, Q8, SP>, grid, S::kThreads, S::kSmem, stream, !std::is_same<SP, SplitArgs>::value, sp);
}

template <class SP>
cudaError_t run_dim(const SP& sp, bool q8, int grid, cudaStream_t stream) {
    if (sp.a.head_dim <= 64) return q8 ? run<64, true>(sp, grid, stream) : run<64, false>(sp, grid, stream);
    if (sp.a.head_dim <= 128) return q8 ? run<128, true>(sp, grid, stream) : run<128, false>(sp, grid, stream);
    return q8 ? run<256, true>(sp, grid, stream) : run<256, false>(sp, grid, stream);
}

}  // namespace

size_t attn_tc_partial_floats(int head_dim) { return partial_floats(kRows, head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256); }

cudaError_t launch_attn_tc(const SplitArgs& sp, bool pass, bool q8, const DeviceInfo& dev, cudaStream_t stream) {
    const AttnArgs& a = sp.a;
    const int tile = a.head_dim <= 128 ? 128 : 64;
    // At least as many units as the batch can have: a CTA for each, where they are few.
    const double reach = std::min(static_cast<double>(a.width) * a.page_size, a.window > 0 ? static_cast<double>(a.window) + a.T : 1e18);
    const double most = static_cast<double>(a.kv_heads) * (a.B + static_cast<double>(a.T) * sp.G / kRows) * (reach / tile + 2 + kFixed);
    const int grid = static_cast<int>(std::min<double>(std::min(dev.sm_count, kMaxTcCtas), most));
    if (!pass) return run_dim(sp, q8, grid, stream);
    const PassArgs args = {sp};
    return run_dim(args, q8, grid, stream);
}

}  // namespace w4
