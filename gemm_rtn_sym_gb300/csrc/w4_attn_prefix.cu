// The pass over prefixes that many rows share: tcgen05 products, one CTA to an
// SM, two warpgroups of 128 row threads in turn.
//
//   S [128 rows, 128 tokens] = Q [rows, D] · Kᵀ    both from shared memory
//   O [128 rows, D]         += P [rows, tokens] · V  P from tensor memory
//
// All rows see all tokens of a prefix, so that nothing is masked but the end of
// the last tile.  A tile is 512 cycles of the tensor cores for S and 1024 for O
// (the weights as two bf16 each, 16 bits: one alone would err as much as the
// result's rounding), at D = 128, and about as long for the threads that hold
// its rows.  With one group of them the two would take turns; so there are
// two, for even and for odd tiles of an item, each with its own S, O and
// statistics: while one group makes its weights, the other's products run.  At
// an item's end their sums meet: a row's two threads share its lane of tensor
// memory, and each writes half of its columns.
//
// Warps 0 to 7 hold the rows, the next ones bring keys and values, the last one
// issues the products.  A stage of the ring is the keys of tile i and the values
// of tile i − 2.  The scores of tile i go where the weights of tile i − 2 were,
// and are issued when the products of those are complete: the order in which
// products are carried out is a promise for those of one shape into one
// accumulator only.  Whole tiles come by TMA, a page (or 128
// tokens of one) and 64 columns at a time, where page sizes divide a tile or
// are multiples of it; an item's end and pages of other sizes come row by row by
// cp.async.  (All rows by cp.async: 1 to 3 % longer.)
// Tensor memory: S of even and of odd tiles from column 0, then the two O.
//
// Format 8: codes are exact as bf16, so the products are those of format 16,
// with the key scales applied to the scores and the value scales to the
// weights.  Codes arrive in slots of their own and eight warps turn them to
// bf16.
//
// The work is the list of (group, head, 128 rows) and their tiles in equal
// pieces over the SMs; parts of items stay where they are, for the join.
//
// Measured.  64 rows of 40 query and 8 key-value heads of 128 behind 16385
// tokens, 67 MB: 42 µs of 60 for all three kernels; 13 are the bytes, 11 the
// products at the measured rates, and 20 the products as they are (each weight
// twice, 320 rows to a head as 384).  Tensor pipe 38 % active, issue 37 %: a tile
// is 3000 cycles, of which the products are 1536, and two groups of rows do not
// hide the rest from one another: their exponentials, roundings and maxima, 640
// instructions to a row at the least, the hand-overs between the three
// kinds of warps, and the pause between a tile's second product and the scores
// that go over its weights (3 µs of the 60; 17 of 121 for 128 rows of 64 heads,
// whose tensor cores have no other pause).  Twelve prefixes of 300 to 8192 tokens
// in format 8, 20 to 40 rows of 64 heads behind each: 70 of 134 µs, bound by
// instructions (issue 53 %), the codes' turn to bf16 among them.
// No faster: the next scores on their way while these are weighed (58.9 for
// 59.4), the joins' work by the CTA that ends an item (25 to 40 µs more), polling
// instead of a suspended wait for the second product (62.1 for 61.4).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda.h>
#include <cudaTypedefs.h>
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

constexpr int kRows = 128, kTile = 128;
constexpr int kRowWarps = 8, kRowThreads = kRowWarps * 32;
constexpr int kFixed = 4;  // an item's fixed cost in tiles
constexpr uint32_t kTmemCols = 512, kColO = 256;

// Waits, as a warp, suspended between tests (polls, which the other kernel's longer stages do not notice, took issue
// slots here: 1 % of the pass); as wait_or_report otherwise.
__device__ __forceinline__ void wait_or_report_suspended(uint32_t bar, uint32_t parity, bool& alive, unsigned* status) {
    if (!alive || __all_sync(~0u, mbar_wait_suspend(bar, parity))) return;
    record_status(status, kStatusTimeout);
    alive = false;
    mbar_wait(bar, parity);
    __syncwarp();
}

template <class S, bool Q8>
__device__ __forceinline__ void fewer_registers() {
    if (Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kOtherRegs));
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// Keys and values as [pages, page_size, heads, head_dim] (or with page_size and heads the other way round) for copies of
// `tokens` tokens of a head, 64 values each; 0: pages of other sizes, copied row by row.
struct Boxes {
    CUtensorMap k, v;
    int tokens;
    bool heads_inside;  // dimension 1 is the head
};

// A matrix descriptor from its lower half (address / 16, leading offset / 16 << 16): 128-byte swizzle, eight rows 1024
// bytes apart.  Issuing is what a thread with 24 products a tile is short of, so that only this half is computed.
__device__ __forceinline__ uint64_t descriptor(uint32_t low) {
    return static_cast<uint64_t>(1024 >> 4 | 1u << 14 | 2u << 29) << 32 | low;
}
static_assert(kRows == kTile, "one offset for queries and keys");

template <int D, bool Q8>
struct Shape {
    // Format 8: whole warpgroups (three warps only make up the last one), so that the rows' can have more registers than
    // the others.  The sum is what the block is launched with, which the launch checks: a thread that asks for more than
    // there are waits for ever.  (81 µs without for 64 rows of 40 heads behind 16385 tokens: 86.  Format 16 has enough.)
    static constexpr int kLoadWarps = Q8 ? 8 : 4, kMmaWarp = kRowWarps + kLoadWarps, kThreads = 32 * (kMmaWarp + (Q8 ? 4 : 1));
    static constexpr int kLaunchRegs = 96, kRowRegs = 144, kOtherRegs = 64;
    static_assert(!Q8 || 2 * kRowRegs + (kLoadWarps / 4 + 1) * kOtherRegs == kThreads / 128 * kLaunchRegs, "all there are");
    static constexpr int kHalf = kTile * D * 2;       // keys or values of a tile
    static constexpr int kStages = Q8 ? 2 : 3;        // of keys and values, what shared memory holds at D = 128
    static constexpr int kQ = kRows * D * 2;
    // Format 8: tiles of codes on their way, in slots of their own.
    static constexpr int kAhead = 2, kRaw = kTile * D, kRawSlots = Q8 ? kAhead + 1 : 0;
    // At least what keeps a second CTA, which would wait for tensor memory, off the SM.
    static constexpr int kNeed = 1024 + kQ + 2 * kStages * kHalf + kRawSlots * kRaw;
    static constexpr int kSmem = kNeed > 120 * 1024 ? kNeed : 120 * 1024;
};

template <int D, bool Q8>
__global__ void __launch_bounds__(Shape<D, Q8>::kThreads, 1) attn_prefix_kernel(const __grid_constant__ PrefixArgs sp, const __grid_constant__ Boxes boxes) {
    using S = Shape<D, Q8>;
    constexpr int TT = kTile, NS = S::kStages, kLoadWarps = S::kLoadWarps, kMmaWarp = S::kMmaWarp;
    extern __shared__ uint8_t smem_raw[];
    // By the tile's group: its scores are there, its weights; a tile's weights have been used; all of an item's products
    // are in O.
    __shared__ __align__(8) uint64_t s_full[NS], s_empty[NS], s_scores[2], s_weights[2], s_used, s_values, s_queries;
    // Format 8, for four tiles: the tokens' key scales (times that of the scores) and value scales.  Where a tile's
    // keys find their stage free, the weights of four tiles before have been used.
    __shared__ __align__(8) uint64_t s_scaled[4];
    __shared__ __align__(16) float s_scale[Q8 ? 4 : 1][2][Q8 ? TT : 4];
    __shared__ float2 s_stats[kRows];  // of a row: the odd tiles' reference and sum, then the factors of both groups' sums
    __shared__ uint32_t s_tmem;
    const AttnArgs& a = sp.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t q_smem = (smem_addr(smem_raw) + 1023) & ~1023u, ring = q_smem + S::kQ;

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_addr(&s_full[i]), 2 * kLoadWarps * 32);
            mbar_init(smem_addr(&s_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&s_scores[i]), 1);
            mbar_init(smem_addr(&s_weights[i]), kRowThreads / 2);
        }
        for (int i = 0; i < 4; ++i) mbar_init(smem_addr(&s_scaled[i]), kLoadWarps * 32);
        mbar_init(smem_addr(&s_used), 1);
        mbar_init(smem_addr(&s_values), 1);
        mbar_init(smem_addr(&s_queries), kRowThreads);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    let_next_start(sp);
    Walk<TT, kRows, kFixed> walk;
    if (!walk.template find<S::kThreads>(sp)) return;
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&s_tmem), kTmemCols);
    if (warp == kRowWarps && lane < 2 && boxes.tokens > 0) asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &boxes.v : &boxes.k));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool alive = true;

    if (warp >= kMmaWarp) {
        // ------------------------------------------------------ products
        fewer_registers<S, Q8>();  // (one instruction for all of a group's warps)
        // A factor below zero turns the queries' signs over.
        const uint32_t qk_idesc = idesc_bf16(TT) | (sp.flip ? 1u << 13 : 0u), pv_idesc = idesc_bf16(D) | 1u << 16;  // B (values) N-major
        Turn stage;
        uint32_t summed[2] = {0, 0}, used = 0, items = 0;  // tiles of each group so far
        for (Item it; warp == kMmaWarp && walk.next(sp, it);) {
            const int tiles = tiles_of<TT>(it);
            wait_or_report_suspended(smem_addr(&s_queries), items++ & 1, alive, a.status);
            // Stage i: the values of tile i − 2, then the keys of tile i, whose scores go where those weights are.
            for (int i = 0; i < tiles + 2; ++i) {
                const int w = i & 1;
                wait_or_report_suspended(smem_addr(&s_full[stage.place]), stage.round, alive, a.status);
                if (i >= 2) wait_or_report_suspended(smem_addr(&s_weights[w]), summed[w]++ & 1, alive, a.status);
                fence_async_smem();  // the copies were made through the generic proxy
                tc_fence_after();
                const uint32_t keys = ring + stage.place * 2 * S::kHalf, vals = keys + S::kHalf;
                if (i >= 2) {
                    if (elect_one()) {
                        // Sixteen tokens' weights: 8 columns of their upper halves, 16 columns further the lower ones.
                        const uint32_t to = tmem + kColO + w * D, weights = tmem + w * TT;
                        const uint32_t low = vals >> 4 | (TT * 128 >> 4) << 16;
#pragma unroll
                        for (int ks = 0; ks < TT / 16; ++ks) {
                            const uint64_t desc = descriptor(low + ks * (2048 >> 4));
                            mma_bf16_tmem_a(to, weights + (ks >> 1) * 32 + (ks & 1) * 8, desc, pv_idesc, 1);
                            mma_bf16_tmem_a(to, weights + (ks >> 1) * 32 + (ks & 1) * 8 + 16, desc, pv_idesc, 1);
                        }
                        if (i < tiles) mma_commit(smem_addr(&s_used));
                    }
                    __syncwarp();
                    if (i < tiles) wait_or_report_suspended(smem_addr(&s_used), used++ & 1, alive, a.status);
                    tc_fence_after();
                }
                if (elect_one()) {
                    if (i < tiles) {
                        const uint32_t to = tmem + w * TT, q_low = q_smem >> 4 | 1u << 16, k_low = keys >> 4 | 1u << 16;
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint32_t off = ((ks >> 2) * kRows * 128 + (ks & 3) * 32) >> 4;
                            mma_bf16(to, descriptor(q_low + off), descriptor(k_low + off), qk_idesc, ks > 0);
                        }
                        mma_commit(smem_addr(&s_scores[w]));
                    }
                    mma_commit(smem_addr(&s_empty[stage.place]));
                    if (i == tiles + 1) mma_commit(smem_addr(&s_values));
                }
                __syncwarp();
                stage.step(NS);
            }
        }
    } else if (warp >= kRowWarps) {
        // -------------------------------------------------------- copies
        fewer_registers<S, Q8>();
        // A warp copies TT / kLoadWarps tokens of each tile; lane l knows token l of them.
        // Format 8: into slots of codes, which the lane that copied them turns to bf16, kAhead half tiles later.
        constexpr int kMine = TT / kLoadWarps, kSub = Q8 ? 1 : kMine / 16, kChunks = D * (Q8 ? 1 : 2) / 16;
        constexpr int kPerPass = 32 / kChunks;  // token rows of one pass of the warp's lanes
        const int my_row = (warp - kRowWarps) * kMine, d_chunks = a.head_dim * (Q8 ? 1 : 2) / 16;
        const int load_c = lane % kChunks, load_r = lane / kChunks;
        Turn stage;
        stage.round = 1;  // the ring's first round finds its stages free
        auto place_of = [&](bool key) { return ring + (2 * stage.place + !key) * S::kHalf; };
        auto begin = [&](bool key) {  // keys come first
            if (key) wait_or_report_suspended(smem_addr(&s_empty[stage.place]), stage.round, alive, a.status);
        };
        auto end = [&](bool key) {
            if (!key) stage.step(NS);
        };
        auto nothing = [&](bool key) {
            begin(key);
            mbar_arrive(smem_addr(&s_full[stage.place]));
            end(key);
        };
        uint32_t scaled = 0;  // tiles whose scales are in shared memory
        const uint32_t raw = ring + 2 * NS * S::kHalf + ((warp - kRowWarps) * kMine * kChunks + lane) * 16;
        int asked = 0, raw_ask = 0, raw_take = 0;
        // What the codes on their way are: keys or values, or none.
        struct Half {
            bool key, any;
        };
        Half way[2] = {};
        // The scales of the lane's token, in the tile found last and in the one before it, as they come: they are moved and
        // converted a stage after they were asked for, so that nothing waits for them.
        struct Scales {
            __nv_bfloat16 k, v;
        };
        const Scales none = {__ushort_as_bfloat16(0), __ushort_as_bfloat16(0)};
        Scales found = none, older = none;
        static_assert(S::kAhead == 2, "two halves on their way");
        // Asks for half a stage of codes (or, past the last, for nothing) and turns that of kAhead before.
        auto half_stage = [&](Half half, long long off) {
            if (half.any) {
                const uint8_t* src = static_cast<const uint8_t*>(half.key ? a.k : a.v) + load_c * 16;
#pragma unroll
                for (int p = 0; p < kMine; p += kPerPass) {
                    const long long o = __shfl_sync(~0u, off, p + load_r);
                    const bool there = o >= 0 && load_c < d_chunks;
                    cp_async16_zfill(raw + raw_ask * S::kRaw + p * kChunks * 16, there ? src + o : static_cast<const uint8_t*>(a.k), there ? 16 : 0);
                }
            }
            cp_async_commit();
            if (++raw_ask == S::kAhead + 1) raw_ask = 0;
            const Half now = way[0];
            way[0] = way[1];
            way[1] = half;
            if (asked < S::kAhead) {
                ++asked;
                return;
            }
            cp_async_wait<S::kAhead>();
            begin(now.key);
            if (now.any) {
                const uint32_t dst = place_of(now.key);
                // A 16-byte chunk of codes makes two of values; lanes in the upper half of 128 bytes of codes write the
                // second one first, so that eight lanes' chunks fall in different banks.
                const int second = D > 64 && (load_c & 4) ? 1 : 0;
#pragma unroll 4
                for (int p = 0; p < kMine; p += kPerPass) {
                    const uint4 w = lds128(raw + raw_take * S::kRaw + p * kChunks * 16);
                    const uint2 x = codes_bf16(w.x), y = codes_bf16(w.y), z = codes_bf16(w.z), u = codes_bf16(w.w);
                    const uint4 lo = make_uint4(x.x, x.y, y.x, y.y), hi = make_uint4(z.x, z.y, u.x, u.y);
                    sts128(dst + place<TT>(my_row + p + load_r, 2 * load_c + second), second ? hi : lo);
                    sts128(dst + place<TT>(my_row + p + load_r, 2 * load_c + (second ^ 1)), second ? lo : hi);
                }
                if (now.key) {
                    const int buffer = scaled++ & 3;
                    if (lane < kMine) {
                        s_scale[Q8 ? buffer : 0][0][Q8 ? my_row + lane : 0] = __bfloat162float(older.k) * sp.scale_log2;
                        s_scale[Q8 ? buffer : 0][1][Q8 ? my_row + lane : 0] = __bfloat162float(older.v);
                    }
                    mbar_arrive(smem_addr(&s_scaled[buffer]));
                }
            }
            if (++raw_take == S::kAhead + 1) raw_take = 0;
            mbar_arrive(smem_addr(&s_full[stage.place]));
            end(now.key);
        };
        for (Item it; walk.next(sp, it);) {
            const int tiles = tiles_of<TT>(it);
            const int* table = a.table + it.b * a.table_stride;
            auto token_of = [&](int i) { return it.tok0 + i * TT + my_row + (lane & (kMine - 1)); };
            auto page_of = [&](int i) {  // page id of the lane's token, −1 outside the piece
                return i < tiles && token_of(i) < it.tok1 ? __ldg(table + sp.page_index(token_of(i))) : -1;
            };
            int page_next = -1;
            long long off = -1, off1 = -1, off2 = -1;  // of the lane's token: in the tile found last, one and two before
            auto find = [&](int i) {
                const int tok = token_of(i), page = page_next;
                page_next = page_of(i + 1);
                off = -1;
                if (tok >= it.tok1) return;
                if (page < 0 || page >= a.pages) {
                    record_status(a.status, kStatusInvalid);
                    return;
                }
                const int in_page = tok - sp.page_index(tok) * a.page_size;
                off = page * a.page_stride + in_page * a.token_stride + it.h * a.head_stride;
                if constexpr (Q8) {
                    const long long at = (static_cast<long long>(page) * a.kv_heads + it.h) * a.page_size + in_page;
                    found.k = a.k_scales[at];
                    found.v = a.v_scales[at];
                }
            };
            // Whole tiles come in boxes, where pages allow it, and an item's end by rows, with zeros behind its last.  Lane
            // l of the warp's has box l / blocks, columns 64 · (l % blocks).
            constexpr int kBlocks = D / 64;
            const int in_boxes = !Q8 && boxes.tokens > 0 ? (it.tok1 - it.tok0) / TT : 0;
            const int per_warp = boxes.tokens <= kMine ? (in_boxes > 0 ? kMine / boxes.tokens : 0) : warp % (boxes.tokens / kMine) == 0;
            const int box_row = my_row + lane / kBlocks * boxes.tokens, block = lane % kBlocks;
            const bool mine = lane / kBlocks < per_warp && 64 * block < a.head_dim;
            auto box_page = [&](int i) { return mine && i < in_boxes ? __ldg(table + sp.page_index(it.tok0 + i * TT + box_row)) : 0; };
            int page0 = 0, page1 = 0, page2 = 0, next_page = box_page(0);  // of this tile, one and two before, and the next
            auto copy_box = [&](bool key, int i, int page) {
                begin(key);
                const uint32_t bar = smem_addr(&s_full[stage.place]);
                if (mine) {
                    if (page < 0 || page >= a.pages) {
                        record_status(a.status, kStatusInvalid);
                        page = -1;  // read as zeros
                    }
                    const int tok = it.tok0 + i * TT + box_row, in_page = tok - sp.page_index(tok) * a.page_size;
                    mbar_arrive_expect_tx(bar, boxes.tokens * 128);
                    tma_load_4d(place_of(key) + block * TT * 128 + box_row * 128, key ? &boxes.k : &boxes.v, 64 * block,
                                boxes.heads_inside ? it.h : in_page, boxes.heads_inside ? in_page : it.h, page, bar);
                } else {
                    mbar_arrive(bar);
                }
                end(key);
            };
            auto copy = [&](bool key, long long from_off) {  // of bf16 rows
                long long off0[kSub];                        // of the first token of each 16
#pragma unroll
                for (int sub = 0; sub < kSub; ++sub) off0[sub] = __shfl_sync(~0u, from_off, 16 * sub);
                const long long mine = kSub == 2 && (lane & 16) ? off0[kSub - 1] : off0[0];
                const bool even = __all_sync(~0u, mine >= 0 && from_off == mine + (lane & 15) * a.token_stride) && d_chunks == kChunks;
                begin(key);
                const uint32_t dst = place_of(key);
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
                        const long long o = __shfl_sync(~0u, from_off, p + load_r);
                        const bool there = o >= 0 && load_c < d_chunks;
                        cp_async16_zfill(dst + place<TT>(my_row + p + load_r, load_c), src + (there ? o + load_c * 8 : 0), there ? 16 : 0);
                    }
                }
                cp_async_arrive(smem_addr(&s_full[stage.place]));
                end(key);
            };
            if (in_boxes < tiles) page_next = page_of(in_boxes);
            for (int i = 0; i < tiles + 2; ++i) {  // keys of tile i, then values of tile i − 2
                off2 = off1, off1 = off;
                page2 = page1, page1 = page0;
                if (i < in_boxes) {
                    page0 = next_page;
                    next_page = box_page(i + 1);
                    copy_box(true, i, page0);
                } else {
                    older = found;
                    found = none;
                    if (i < tiles) find(i);
                    if constexpr (Q8)
                        half_stage({true, i < tiles}, off);
                    else if (i < tiles)
                        copy(true, off);
                    else
                        nothing(true);
                }
                if (i >= 2 && i - 2 < in_boxes) {
                    copy_box(false, i - 2, page2);
                } else {
                    if constexpr (Q8)
                        half_stage({false, i >= 2}, off2);
                    else if (i >= 2)
                        copy(false, off2);
                    else
                        nothing(false);
                }
            }
        }
        if constexpr (Q8) {
            if (asked > 0) {
#pragma unroll 1
                for (int i = 0; i < S::kAhead; ++i) half_stage({i % 2 == 0, false}, 0);
            }
        }
        cp_async_wait_all();
    } else {
        // ------------------------------------------- a row in every thread
        if (Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRowRegs));
        auto rows_sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kRowThreads) : "memory"); };
        const int group = warp >> 2, own_row = tid & (kRows - 1);
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16), scores = lanes + group * TT, out = lanes + kColO + group * D;
        uint32_t tile = 0, four = 0, items = 0;  // tiles of the group so far; of both; items
        // The queries of an item: a row by D / 8 lanes.
        auto ask = [&](const Item& n) {
            constexpr int kChunks = D / 8, kPerPass = kRowThreads / kChunks;
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
            const int tiles = tiles_of<TT>(it);
            const int row = it.row0 + own_row, j = sp.over_G(row);
            const bool live = row < it.rows;
            {
                uint32_t zero[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) zero[x] = 0;
#pragma unroll
                for (int c = 0; c < D; c += 32) tmem_st32(out + c, zero);
                tmem_wait_st();
            }
            cp_async_wait_all();
            fence_async_smem();
            tc_fence_before();
            mbar_arrive(smem_addr(&s_queries));
            float m = -INFINITY, l = 0.f;  // reference score, unscaled (format 8: to base 2); sum of the weights
            const float unit = Q8 ? 1.f : sp.scale_log2;
            for (int i = group; i < tiles; i += 2, ++tile) {
                const int there = it.tok1 - it.tok0 - i * TT;  // columns that are tokens
                wait_or_report_suspended(smem_addr(&s_scores[group]), tile & 1, alive, a.status);
                tc_fence_after();
                const uint32_t buffer = (four + i) & 3;
                if (Q8) wait_or_report_suspended(smem_addr(&s_scaled[buffer]), (four + i) >> 2 & 1, alive, a.status);
                const float(*const scale)[Q8 ? TT : 4] = s_scale[Q8 ? buffer : 0];
                // A tile's scores are read twice, 32 at a time in rolled loops: held in 128 registers in between, with all
                // loops unrolled, they cost as much in instructions that the caches do not have (a fifth of all stalls).
                auto hide = [&](uint32_t(&u)[32], int c) {  // (in a loop of its own: selects in every tile cost 7 %)
                    if (there < TT)
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (32 * c + x >= there) u[x] = 0xFF800000u;  // −∞
                };
                // Factors of two tokens' scores to base 2.
                auto units = [&](int column) { return Q8 ? *reinterpret_cast<const uint64_t*>(&scale[0][Q8 ? column : 0]) : two(unit, unit); };
                // ---- reference
                float most[4] = {m, -INFINITY, -INFINITY, -INFINITY};
                auto larger = [&](const uint32_t(&u)[32]) {
#pragma unroll
                    for (int x = 0; x < 32; x += 8)
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            most[y] = fmaxf(most[y], fmaxf(__uint_as_float(u[x + 2 * y]), __uint_as_float(u[x + 2 * y + 1])));
                };
#pragma unroll 2
                for (int c = 0; c < TT / 32; ++c) {
                    uint32_t u[32];
                    tmem_ld32(scores + 32 * c, u);
                    if (Q8)
#pragma unroll
                        for (int x = 0; x < 32; x += 2) {
                            const uint64_t s = mul2(two(__uint_as_float(u[x]), __uint_as_float(u[x + 1])), units(32 * c + x));
                            u[x] = __float_as_uint(first_of(s));
                            u[x + 1] = __float_as_uint(second_of(s));
                        }
                    hide(u, c);
                    larger(u);
                }
                const float grown = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
                const float by = (grown - m) * unit;
                if (__any_sync(~0u, by > 8.f)) {
                    const float keep = m == -INFINITY ? 0.f : ex2(-by);
                    if (i >= 2) {  // (this tile's scores were issued after the products before, and are there)
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t u[16];
                            tmem_ld16(out + c, u);
#pragma unroll
                            for (int x = 0; x < 16; ++x) u[x] = __float_as_uint(__uint_as_float(u[x]) * keep);
                            tmem_st16(out + c, u);
                        }
                        tmem_wait_st();
                    }
                    l *= keep;
                    m = grown;
                }
                const float ref = m == -INFINITY ? 0.f : m * unit;
                // ---- weights, over the scores: of 32 tokens the upper halves in 16 columns, then the lower ones
                const uint64_t from = two(-ref, -ref);
                uint64_t sums[2] = {two(l, 0.f), 0};
                auto weigh = [&](const uint32_t(&u)[32], int c) {
                    uint32_t w[32];
#pragma unroll
                    for (int x = 0; x < 32; x += 2) {
                        uint64_t s = two(__uint_as_float(u[x]), __uint_as_float(u[x + 1]));
                        if (!Q8) s = fma2(s, units(0), from);
                        uint64_t p = two(ex2(first_of(s)), ex2(second_of(s)));
                        sums[x >> 1 & 1] = add2(sums[x >> 1 & 1], p);
                        if (Q8) p = mul2(p, *reinterpret_cast<const uint64_t*>(&scale[1][Q8 ? 32 * c + x : 0]));
                        // Both halves cut off, not rounded (roundings to bf16 would share the exponentials' slow
                        // pipe): the lower ones take what the upper ones leave, to 16 bits in all, at most 2⁻¹⁵ and
                        // on the average 2⁻¹⁷ of the weight too low.
                        const uint32_t u0 = __float_as_uint(first_of(p)), u1 = __float_as_uint(second_of(p));
                        const uint64_t left = add2(p, two(__uint_as_float((u0 & 0xFFFF0000u) ^ 0x80000000u), __uint_as_float((u1 & 0xFFFF0000u) ^ 0x80000000u)));
                        w[x >> 1] = __byte_perm(u0, u1, 0x7632);
                        w[16 + (x >> 1)] = __byte_perm(__float_as_uint(first_of(left)), __float_as_uint(second_of(left)), 0x7632);
                    }
                    tmem_st32(scores + 32 * c, w);
                };
#pragma unroll 2
                for (int c = 0; c < TT / 32; ++c) {
                    uint32_t u[32];
                    tmem_ld32(scores + 32 * c, u);
                    if (Q8)
#pragma unroll
                        for (int x = 0; x < 32; x += 2) {
                            const uint64_t s = fma2(two(__uint_as_float(u[x]), __uint_as_float(u[x + 1])), units(32 * c + x), from);
                            u[x] = __float_as_uint(first_of(s));
                            u[x + 1] = __float_as_uint(second_of(s));
                        }
                    hide(u, c);
                    weigh(u, c);
                }
                l = (first_of(sums[0]) + second_of(sums[0])) + (first_of(sums[1]) + second_of(sums[1]));
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_addr(&s_weights[group]));
            }
            four += tiles;
            // ---- the two groups' sums
            wait_or_report_suspended(smem_addr(&s_values), items++ & 1, alive, a.status);
            tc_fence_after();
            tc_fence_before();
            if (group == 1) s_stats[own_row] = make_float2(m * unit, l);
            rows_sync();
            tc_fence_after();
            float top = 0.f, sum = 0.f, by_even, by_odd;  // (top and sum: of the even group's threads)
            if (group == 0) {
                const float2 odd = s_stats[own_row];
                top = fmaxf(m * unit, odd.x);
                const float ref = top == -INFINITY ? 0.f : top;
                by_even = ex2(m * unit - ref);
                by_odd = ex2(odd.x - ref);
                sum = l * by_even + odd.y * by_odd;
                s_stats[own_row] = make_float2(by_even, by_odd);
            }
            rows_sync();
            if (group == 1) by_even = s_stats[own_row].x, by_odd = s_stats[own_row].y;
            const bool whole = it.whole();
            const Parts<kRows, D> parts(sp, walk, it, kFixed);
            const size_t at_row = static_cast<size_t>(it.start + j) * a.q_heads + it.h * sp.G + row - j * sp.G;
            // A part of an item is [reference and sum of each row], then D values of each; the item's first part says where
            // they are.
            const int k = static_cast<int>(blockIdx.x) - parts.first;
            float* const part = parts.at(k);
            if (live && group == 0) {
                if (!whole) reinterpret_cast<float2*>(part)[own_row] = make_float2(top, fminf(sum, 3e38f));
                if (k == 0) a.sums[at_row] = make_float4(top, fminf(sum, 3e38f), __int_as_float(whole ? 0 : parts.count), __int_as_float(parts.first << 8 | own_row));
            }
            // A warp's 32 rows go out through its part of the queries' place, some columns at a time, so that a row's lie side
            // by side (16-byte chunks of eight rows in different banks).
            constexpr int kCols = D / 4, kPieces = kCols / 4, kRowsAtOnce = 32 / kPieces;
            float* const to = whole ? a.sum_values + at_row * a.head_dim : part + 2 * kRows + own_row * D;
            const uint32_t corner = q_smem + warp * 32 * kCols * 4;
            auto chunk = [&](int r, int q) { return corner + (r * kPieces + (q ^ (r & (kPieces - 1)))) * 16; };
#pragma unroll 1
            for (int c = group * (D / 2); c < (group + 1) * (D / 2); c += kCols) {
                uint32_t u[kCols / 16][16], v[kCols / 16][16];
#pragma unroll
                for (int y = 0; y < kCols / 16; ++y) {
                    tmem_ld16_async(lanes + kColO + c + 16 * y, u[y]);
                    tmem_ld16_async(lanes + kColO + D + c + 16 * y, v[y]);
                }
                tmem_wait_ld();
#pragma unroll
                for (int y = 0; y < kCols / 16; ++y) {
                    reg_fence16(u[y]);
                    reg_fence16(v[y]);
                    auto joined = [&](int x) { return __float_as_uint(fmaf(__uint_as_float(v[y][x]), by_odd, __uint_as_float(u[y][x]) * by_even)); };
#pragma unroll
                    for (int x = 0; x < 16; x += 4) sts128(chunk(lane, 4 * y + x / 4), make_uint4(joined(x), joined(x + 1), joined(x + 2), joined(x + 3)));
                }
                __syncwarp();
                const int q = lane % kPieces, col = c + 4 * q;
#pragma unroll
                for (int r = 0; r < 32; r += kRowsAtOnce) {
                    const int from = r + lane / kPieces;
                    float* const row_to = reinterpret_cast<float*>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(to), from));
                    const uint4 w = lds128(chunk(from, q));
                    if (it.row0 + (own_row & ~31) + from < it.rows && col < a.head_dim) *reinterpret_cast<uint4*>(row_to + col) = w;
                }
                __syncwarp();
            }
            tc_fence_before();
            rows_sync();  // the sums are read: the next item's may begin
            tc_fence_after();
            Item after;
            more = walk.next(sp, after);
            if (more) ask(after);
            it = after;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 found = [] {
        cudaDriverEntryPointQueryResult q;
        void* fn = nullptr;
        const bool there = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                           q == cudaDriverEntryPointSuccess;
        return there ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn) : nullptr;
    }();
    return found;
}

// Boxes of the cache's pages, where they serve: whole rows of 64 values, and tiles of whole pages or pages of whole
// tiles, at eight rows or more a box (what the swizzle repeats after).  Values past head_dim and pages out of range
// read as zeros.
Boxes boxes_of(const AttnArgs& a) {
    Boxes b = {};
    const int P = a.page_size, tokens = P % kTile == 0 ? kTile : P < kTile && kTile % P == 0 ? P : 0;
    if (tokens < 8 || a.head_dim < 64 || !encoder()) return b;
    // (a dimension of one has no stride of its own)
    const cuuint64_t heads = a.kv_heads > 1 ? a.head_stride * 2 : a.head_dim * 2, places = a.token_stride * 2, pages = a.pages > 1 ? a.page_stride * 2 : 16;
    b.heads_inside = heads <= places;
    const cuuint64_t H = a.kv_heads, size = P;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.head_dim), b.heads_inside ? H : size, b.heads_inside ? size : H, static_cast<cuuint64_t>(a.pages)};
    const cuuint64_t strides[3] = {b.heads_inside ? heads : places, b.heads_inside ? places : heads, pages};
    const cuuint32_t n = tokens, box[4] = {64u, b.heads_inside ? 1u : n, b.heads_inside ? n : 1u, 1u}, each[4] = {1, 1, 1, 1};
    for (int i = 0; i < 2; ++i)
        if (encoder()(i ? &b.v : &b.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(i ? a.v : a.k), dims, strides, box, each,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return b;  // (strides past what a map can say: row by row)
    b.tokens = tokens;
    return b;
}

template <int D, bool Q8>
cudaError_t run(const SplitArgs& sp, int grid, cudaStream_t stream) {
    using S = Shape<D, Q8>;
    static std::atomic<bool> ready[kMaxDevices];  // the kernel may use its shared memory on this device
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    if (err != cudaSuccess) return err;
    if (!ready[device & (kMaxDevices - 1)].load(std::memory_order_relaxed)) {
        cudaFuncAttributes attributes;
        err = cudaFuncGetAttributes(&attributes, attn_prefix_kernel<D, Q8>);
        if (err != cudaSuccess) return err;
        if (Q8 && attributes.numRegs != S::kLaunchRegs) return cudaErrorInvalidConfiguration;
        err = cudaFuncSetAttribute(attn_prefix_kernel<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (err != cudaSuccess) return err;
        ready[device & (kMaxDevices - 1)].store(true, std::memory_order_relaxed);
    }
    return launch_pass(attn_prefix_kernel<D, Q8>, grid, S::kThreads, S::kSmem, stream, true, PrefixArgs{sp}, Q8 ? Boxes{} : boxes_of(sp.a));
}

// -------------------------------------------------------------------- join
constexpr int kJoinWarps = 4, kJoinBatch = 8;

// One warp to a row: its own tokens' sums, and those of its prefix, from
// wherever they are, on one reference, into its output.  (The CTA that
// finishes an item last, as in the other kernels, would read its parts alone:
// 19 of 66 KB where one prefix's 8 heads are shared by 152 SMs.)  2 of the 60
// µs and 9 of the 134 above: 2560 rows of 128, each in about 7 parts.
template <int V>  // float4 of a lane: head_dim ≤ 128 · V
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(const __grid_constant__ JoinArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long first = a.starts ? min(max(a.starts[0], 0), a.T) : 0, end = a.starts ? min(max(a.starts[a.B], 0), a.T) : a.T;
    const long long row = (first * a.q_heads) + static_cast<long long>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
    if (row >= end * a.q_heads) return;
    const float4 own = __ldcg(a.own + row);
    const float4 prefix = __ldcg(a.prefix + row);
    const int kind = __float_as_int(own.z);
    const int token = static_cast<int>(row / a.q_heads), head = static_cast<int>(row - static_cast<long long>(token) * a.q_heads);
    float4 v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int col = 4 * (lane + 32 * i);
        v[i] = col < a.head_dim ? __ldcg(reinterpret_cast<const float4*>(a.own_values + row * a.head_dim + col)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float m = own.x, l = own.y;
    auto add = [&](float factor, const float* from) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int col = 4 * (lane + 32 * i);
            if (col >= a.head_dim) continue;
            const float4 u = __ldcg(reinterpret_cast<const float4*>(from + col));
            v[i] = make_float4(fmaf(factor, u.x, v[i].x), fmaf(factor, u.y, v[i].y), fmaf(factor, u.z, v[i].z), fmaf(factor, u.w, v[i].w));
        }
    };
    auto rebase = [&](float to) {  // from reference m to `to`, which is at least as large
        const float ref = to == -INFINITY ? 0.f : to, keep = ex2(m - ref);
        l *= keep;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = make_float4(v[i].x * keep, v[i].y * keep, v[i].z * keep, v[i].w * keep);
        m = to;
        return ref;
    };
    if (kind == kRowShared) {
        // (Where starts fall, nobody may have written the row's prefix: no part that could not be is read.)
        const int at = __float_as_int(prefix.w), in_tile = at & (kRows - 1), first_piece = at >> 8;
        const int said = __float_as_int(prefix.z), count = said > 0 && first_piece >= 0 && said <= a.pieces - first_piece ? said : 0;
        if (count == 0) {
            const float ref = rebase(fmaxf(m, prefix.x)), f = ex2(prefix.x - ref);
            l = fmaf(f, prefix.y, l);
            add(f, a.prefix_values + row * a.head_dim);
        }
        // Part k: the second of piece `first`, the first of those after it.
        auto part = [&](int k) { return a.partial + (2 * static_cast<size_t>(first_piece + k) + (k == 0)) * a.part_floats; };
        for (int k0 = 0; k0 < count; k0 += 32) {
            const int n = min(32, count - k0);
            const float2 stats = lane < n ? __ldcg(reinterpret_cast<const float2*>(part(k0 + lane)) + in_tile) : make_float2(-INFINITY, 0.f);
            float top = stats.x;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
            const float ref = rebase(fmaxf(m, top)), f = ex2(stats.x - ref);
            float sum = f * stats.y;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
            l += sum;
#pragma unroll kJoinBatch
            for (int k = 0; k < n; ++k) add(__shfl_sync(~0u, f, k), part(k0 + k) + 2 * kRows + in_tile * a.D);
        }
    }
    const float f = 1.f / l;
    __nv_bfloat16* const to = a.out.data + token * a.out.token_stride + head * a.out.head_stride;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int col = 4 * (lane + 32 * i);
        if (col < a.head_dim)
            *reinterpret_cast<uint2*>(to + col) = kind == kRowEmpty ? make_uint2(0, 0)
                                                                    : make_uint2(pack_bf16(v[i].x * f, v[i].y * f), pack_bf16(v[i].z * f, v[i].w * f));
    }
}

}  // namespace

cudaError_t launch_attn_join(JoinArgs a, cudaStream_t stream) {
    a.D = a.head_dim <= 64 ? 64 : a.head_dim <= 128 ? 128 : 256;
    a.part_floats = partial_floats(kRows, a.D);
    const long long rows = static_cast<long long>(a.T) * a.q_heads;
    const unsigned grid = static_cast<unsigned>((rows + kJoinWarps - 1) / kJoinWarps);
    return launch_pass(a.head_dim <= 128 ? attn_join_kernel<1> : attn_join_kernel<2>, static_cast<int>(grid), 32 * kJoinWarps, 0, stream, true, a);
}

cudaError_t launch_attn_prefix(const SplitArgs& sp, bool q8, const DeviceInfo& dev, cudaStream_t stream) {
    const AttnArgs& a = sp.a;
    // At least as many units as the batch can have: a CTA for each, where they are few.
    const double reach = static_cast<double>(a.width) * a.page_size;
    const double most = static_cast<double>(a.kv_heads) * (a.B + static_cast<double>(a.T) * sp.G / kRows) * (reach / kTile + 2 + kFixed);
    const int grid = static_cast<int>(std::min<double>(std::min(dev.sm_count, kMaxTcCtas), most));
    if (a.head_dim <= 64) return q8 ? run<64, true>(sp, grid, stream) : run<64, false>(sp, grid, stream);
    return q8 ? run<128, true>(sp, grid, stream) : run<128, false>(sp, grid, stream);
}

}  // namespace w4
