// What the two kernels of attention over the paged cache share: the list of
// work and its pieces, and the joining of items that several CTAs work on.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "w4_device.cuh"
#include "w4_kv.h"

namespace w4 {

constexpr int kJoinGroup = 16;          // parts of an item that are joined at once
constexpr int kMaxLength = 0x7fff0000;  // token numbers a little past a length stay below 2³¹
constexpr int kMaxDevices = 64;         // as many as the library knows (device_info refuses others)
constexpr int kMaxCtas = 512;           // bounds the workspace,
constexpr int kMaxTcCtas = 160;         // and that of the tensor-core kernel, which has one CTA on an SM (of 152)
// Format 8's value scales from here on (2⁻¹⁰⁰): with smaller ones, and for zero, this one stands in.  It has a
// logarithm, the codes of a zero scale are zero, and its inverse times weights of at most 2⁸ can be summed over 2²⁰
// tokens of one warp's stream (tokens of larger scales, where there are any, put the reference up).
constexpr float kLeastScale = 7.888609052210118e-31f;

// The weights' reference and their sum, ROWS of each, then ROWS rows of D values.
__host__ __device__ constexpr size_t partial_floats(int rows, int D) { return static_cast<size_t>(rows) * (2 + D); }

struct SplitArgs {
    AttnArgs a;
    unsigned long long* arrived;  // [2][kMaxCtas] parts there of a group, groups there of an item
    float* partial;               // [kMaxCtas or kMaxTcCtas][2][partial_floats]
    int G;                        // query heads per key-value head
    uint32_t G_mul;               // divide_by(G)
    int G_shift;
    int rows_each;                // rows of each request, where starts is null
    float scale_log2;             // |scale| · log2(e)
    uint32_t flip;                // sign bits of a pair of queries to turn over: scale < 0

    __device__ __forceinline__ int over_G(int r) const { return static_cast<int>((static_cast<uint64_t>(r) * G_mul) >> G_shift); }
    __device__ __forceinline__ int page_index(int token) const {  // token / page_size
        return static_cast<int>((static_cast<uint64_t>(token) * a.page_mul) >> a.page_shift);
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// --------------------------------------------------------------- work list
// A request's part of the work: rows and tokens, clipped to what is there.
struct Request {
    int start, n;     // token rows
    int len;          // tokens in the cache
    int low;          // first token that any row sees
    int tiles;        // tiles of TILE tokens from the one of `low`
    int row_tiles;    // of ROWS rows (new tokens × query heads per key-value head)
};

template <int TILE, int ROWS>
__device__ __forceinline__ Request request(const SplitArgs& sp, int b) {
    const AttnArgs& a = sp.a;
    Request r;
    const int len = a.lens[b];
    if (a.starts) {
        const int T = static_cast<int>(a.T);
        r.start = min(max(a.starts[b], 0), T);
        r.n = min(max(a.starts[b + 1], r.start), T) - r.start;
    } else {
        r.n = sp.rows_each;
        r.start = b * r.n;
    }
    const int most = static_cast<int>(min(static_cast<long long>(a.width) * a.page_size, static_cast<long long>(kMaxLength)));
    if (len < 0 || len > most) record_status(a.status, kStatusInvalid);
    r.len = min(max(len, 0), most);
    const long long low = a.window > 0 ? static_cast<long long>(r.len) - r.n - a.window + 1 : 0;
    r.low = static_cast<int>(max(low, 0ll));
    // A request without tokens still has its rows of zeros to write: one tile.
    r.tiles = max(1, (r.len + TILE - 1) / TILE - r.low / TILE);
    r.row_tiles = (r.n * sp.G + ROWS - 1) / ROWS;
    return r;
}

// Units of work of a request: each item (head, row tile) counts FIXED units
// and then one for each of its tiles.
template <int FIXED>
__device__ __forceinline__ long long units(const AttnArgs& a, const Request& r) {
    return static_cast<long long>(a.kv_heads) * r.row_tiles * (r.tiles + FIXED);
}

__device__ __forceinline__ long long quotient(long long x, int y) {
    return x >> 32 ? static_cast<long long>(static_cast<unsigned long long>(x) / static_cast<unsigned>(y))
                   : static_cast<long long>(static_cast<unsigned>(x) / static_cast<unsigned>(y));
}

// How `total` units are cut into n pieces: the first `longer` of them have one
// unit more than the others' `size`.
struct Cut {
    long long size, longer;

    __device__ __forceinline__ void set(long long total, int n) {
        size = quotient(total, n);
        longer = total - size * n;
    }
    __device__ __forceinline__ long long begin(int p) const { return p * size + min(static_cast<long long>(p), longer); }
    __device__ __forceinline__ int piece(long long unit) const {  // that a unit lies in
        const long long head = longer * (size + 1);
        return static_cast<int>(unit < head ? quotient(unit, static_cast<int>(size) + 1)
                                            : longer + quotient(unit - head, static_cast<int>(size)));
    }
};

// A piece's part of an item: tokens [tok0, tok1), tiles [tile0, tile1) of
// `tiles`, for the rows from row0 on (of `rows`) of head h of request b.
struct Item {
    int b, h, row0, rows;
    int start, n, len;
    int tok0, tok1;
    int tile0, tile1, tiles;
    long long unit;  // the item's first

    __device__ __forceinline__ bool whole() const { return tile0 == 0 && tile1 == tiles; }
};

// Walks the items of a CTA's piece.
template <int TILE, int ROWS, int FIXED>
struct Walk {
    Cut cut;
    long long at, end;  // units of the piece
    long long before;   // units of the requests before b
    int b;
    bool known;         // rq is request b
    Request rq;

    // The total work, and the request that the CTA's piece begins in: each
    // thread sums a stretch of the requests, then one scan over the threads.
    // False (for the whole CTA) where there is no piece.
    template <int THREADS>
    __device__ __forceinline__ bool find(const SplitArgs& sp) {
        __shared__ long long s_sum[THREADS / 32];
        __shared__ long long s_before;
        __shared__ int s_at;
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = sp.a.B;
        const int per = (B + THREADS - 1) / THREADS;
        long long own = 0;
        for (int i = tid * per; i < min((tid + 1) * per, B); ++i) own += units<FIXED>(sp.a, request<TILE, ROWS>(sp, i));
        long long sum = own;
        for (int d = 1; d < 32; d <<= 1) {
            const long long v = __shfl_up_sync(~0u, sum, d);
            if (lane >= d) sum += v;
        }
        if (lane == 31) s_sum[warp] = sum;
        __syncthreads();
        long long total = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) sum += s_sum[w];
            total += s_sum[w];
        }
        cut.set(total, gridDim.x);
        at = cut.begin(blockIdx.x);
        end = cut.begin(blockIdx.x + 1);
        if (at >= end) return false;
        if (at >= sum - own && at < sum) {
            long long first = sum - own;
            int i = tid * per;
            for (const int stop = min(i + per, B) - 1; i < stop; ++i) {
                const long long w = units<FIXED>(sp.a, request<TILE, ROWS>(sp, i));
                if (at < first + w) break;
                first += w;
            }
            s_at = i;
            s_before = first;
        }
        __syncthreads();
        b = s_at;
        before = s_before;
        known = false;
        return true;
    }

    __device__ __forceinline__ bool next(const SplitArgs& sp, Item& s) {
        while (at < end && b < sp.a.B) {
            if (!known) rq = request<TILE, ROWS>(sp, b);
            known = true;
            const long long mine = units<FIXED>(sp.a, rq);
            if (at >= before + mine) {
                before += mine;
                ++b;
                known = false;
                continue;
            }
            const int weight = rq.tiles + FIXED;
            const int line = static_cast<int>(quotient(at - before, weight));
            s.unit = before + static_cast<long long>(line) * weight;
            s.tile0 = max(0, static_cast<int>(at - s.unit) - FIXED);
            s.tile1 = static_cast<int>(min(static_cast<long long>(weight), end - s.unit)) - FIXED;
            at = s.unit + weight;
            if (s.tile1 <= s.tile0) continue;  // the piece ends in the item's fixed units
            s.b = b;
            s.h = rq.row_tiles == 1 ? line : line / rq.row_tiles;
            s.row0 = (line - s.h * rq.row_tiles) * ROWS;
            s.rows = rq.n * sp.G;
            s.start = rq.start;
            s.n = rq.n;
            s.len = rq.len;
            s.tiles = rq.tiles;
            const int low_tile = rq.low / TILE;
            s.tok0 = max(rq.low, (low_tile + s.tile0) * TILE);
            s.tok1 = static_cast<int>(min(static_cast<long long>(rq.len), (low_tile + s.tile1) * static_cast<long long>(TILE)));
            return true;
        }
        return false;
    }
};

// ------------------------------------------------------------------- output
// n values of a row's output from column col on: `v` times 1 / `l`.  A row that
// sees nothing is zeros; one whose scores are all −∞ has no value (0 / 0).
__device__ __forceinline__ void put_row(const SplitArgs& sp, const Item& it, int row, int col, const float* v, int n, float l) {
    const int j = sp.over_G(row);
    const bool none = it.len - it.n + j < 0;
    const float f = 1.f / l;
    __nv_bfloat16* to = sp.a.out.data + (it.start + j) * sp.a.out.token_stride +
                        (it.h * sp.G + row - j * sp.G) * sp.a.out.head_stride + col;
    for (int x = 0; x < n; x += 2) *reinterpret_cast<uint32_t*>(to + x) = none ? 0u : pack_bf16(v[x] * f, v[x + 1] * f);
}

// Counts an arrival at `word`; true for the last of `need`.  The upper 48 bits
// mark a word that counts, and the last arrival leaves the count 0, for the
// next launch; a word without the mark (what the workspace held before its
// first use) counts as none.  What the CTA wrote before its barrier is then
// visible to the CTA of the last arrival.
constexpr unsigned long long kMark = 0x77346B765F61ull << 16;

__device__ __forceinline__ bool arrive(unsigned long long* word, int need) {
    __threadfence();
    unsigned long long seen = atomicAdd(word, 1ull);
    bool counted = (seen & ~0xFFFFull) == kMark;
    int count = static_cast<int>(seen & 0xFFFF) + 1;
    if (!counted) {
        ++seen;
        do {
            count = (seen & ~0xFFFFull) == kMark ? static_cast<int>(seen & 0xFFFF) + 1 : 1;
            const unsigned long long prev = atomicCAS(word, seen, kMark | count);
            counted = prev == seen;
            seen = prev;
        } while (!counted);
    }
    if (count != need) return false;
    __threadfence();
    atomicExch(word, kMark);
    return true;
}

// The parts of an item that several pieces share: piece `first` (which has its
// first tile) and those after it, `count` in all.  A piece's first item leaves
// its sums in slot 0, its last in slot 1.
template <int ROWS, int D>
struct Parts {
    float* partial;
    int first, count;

    template <class W>
    __device__ __forceinline__ Parts(const SplitArgs& sp, const W& walk, const Item& it, int fixed) : partial(sp.partial) {
        first = it.whole() ? static_cast<int>(blockIdx.x) : walk.cut.piece(it.unit + fixed);
        count = it.whole() ? 1 : walk.cut.piece(it.unit + fixed + it.tiles - 1) - first + 1;
    }

    __device__ __forceinline__ float* at(int k) const {
        return partial + (2 * static_cast<size_t>(first + k) + (k == 0)) * partial_floats(ROWS, D);
    }

    // A warp (number `warp` of WARPS) joins NP parts of 16 / NP rows at a time, all loads at once: parts k0, k0 +
    // step, ... (n of them) into the output or into part k0.
    template <int WARPS, int NP>
    __device__ __forceinline__ void join_rows(const SplitArgs& sp, const Item& it, int warp, int lane, int k0, int n, int step, bool last) const {
        constexpr int NR = 16 / NP, V = D / 32;  // V neighbouring values of a lane
        const int y_lane = (lane & 15) / NP, i_lane = lane & (NP - 1);
        for (int r = warp * NR; r < ROWS && it.row0 + r < it.rows; r += WARPS * NR) {
            float mm = -INFINITY, ll = 0.f, v[NR][V];  // mm, ll: of the lane's row
#pragma unroll
            for (int y = 0; y < NR; ++y)
#pragma unroll
                for (int x = 0; x < V; ++x) v[y][x] = 0.f;
            for (int i0 = 0; i0 < n; i0 += NP) {
                const bool there = i0 + i_lane < n;
                const float* mine = at(k0 + min(i0 + i_lane, n - 1) * step) + r + y_lane;
                const float pm = there ? __ldcg(mine) : -INFINITY, pl = __ldcg(mine + ROWS);
                float w[NR][NP][V];
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const float* p = at(k0 + min(i0 + i, n - 1) * step) + 2 * ROWS + r * D + lane * V;
#pragma unroll
                    for (int y = 0; y < NR; ++y)
                        if constexpr (V == 2) {
                            const float2 f = __ldcg(reinterpret_cast<const float2*>(p + y * D));
                            w[y][i][0] = f.x, w[y][i][1] = f.y;
                        } else {
#pragma unroll
                            for (int x = 0; x < V; x += 4) {
                                const float4 f = __ldcg(reinterpret_cast<const float4*>(p + y * D + x));
                                w[y][i][x] = f.x, w[y][i][x + 1] = f.y, w[y][i][x + 2] = f.z, w[y][i][x + 3] = f.w;
                            }
                        }
                }
                float nm = fmaxf(mm, pm);
#pragma unroll
                for (int d = 1; d < NP; d <<= 1) nm = fmaxf(nm, __shfl_xor_sync(~0u, nm, d));
                const float rm = nm == -INFINITY ? 0.f : nm, keep = ex2(mm - rm), f = there ? ex2(pm - rm) : 0.f;
                float fl = there ? f * pl : 0.f;
#pragma unroll
                for (int d = 1; d < NP; d <<= 1) fl += __shfl_xor_sync(~0u, fl, d);
                ll = ll * keep + fl;
                mm = nm;
#pragma unroll
                for (int y = 0; y < NR; ++y) {
                    const float k = __shfl_sync(~0u, keep, y * NP);
#pragma unroll
                    for (int x = 0; x < V; ++x) v[y][x] *= k;
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        const float fi = __shfl_sync(~0u, f, y * NP + i);
#pragma unroll
                        for (int x = 0; x < V; ++x) v[y][x] = i0 + i < n ? fmaf(fi, w[y][i][x], v[y][x]) : v[y][x];
                    }
                }
            }
#pragma unroll
            for (int y = 0; y < NR; ++y) {
                const float l_row = __shfl_sync(~0u, ll, y * NP), m_row = __shfl_sync(~0u, mm, y * NP);
                if (it.row0 + r + y >= it.rows) continue;
                if (last) {
                    if (lane * V < sp.a.head_dim) put_row(sp, it, it.row0 + r + y, lane * V, v[y], V, l_row);
                } else {
                    float* to = at(k0);
                    if (lane == 0) to[r + y] = m_row, to[ROWS + r + y] = fminf(l_row, 3e38f);
#pragma unroll
                    for (int x = 0; x < V; ++x) to[2 * ROWS + (r + y) * D + lane * V + x] = v[y][x];
                }
            }
        }
    }

    // After this CTA has left its part: the last part of a group of sixteen to get here joins the group, the last
    // group the item.  `sync` is a barrier of the warps that take part (thread 0 among them), `s_last` shared by them;
    // `join` (parts k0, k0 + step, ..., n of them, into the output if `last`, else into part k0) is called by all.
    template <class Sync, class Join>
    __device__ __forceinline__ void finish(const SplitArgs& sp, bool& s_last, Sync sync, Join join) const {
        const int own = static_cast<int>(blockIdx.x) - first;
        const int k0 = own / kJoinGroup * kJoinGroup, in_group = min(kJoinGroup, count - k0), groups = (count + kJoinGroup - 1) / kJoinGroup;
        if (in_group > 1) {
            if (threadIdx.x == 0) s_last = arrive(sp.arrived + first + k0, in_group);
            sync();
            const bool last = s_last;
            if (last) join(k0, in_group, 1, groups == 1);
            sync();
            if (!last) return;
        }
        if (groups > 1) {
            if (threadIdx.x == 0) s_last = arrive(sp.arrived + kMaxCtas + first, groups);
            sync();
            if (s_last) join(0, groups, kJoinGroup, true);
            sync();
        }
    }
};

}  // namespace w4
