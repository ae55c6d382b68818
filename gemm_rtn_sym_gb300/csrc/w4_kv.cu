// Paged key-value cache: block tables and slots from request lengths, and
// rotary positions with the new tokens' rows written to the cache.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "w4_device.cuh"
#include "w4_kv.h"

namespace w4 {
namespace {

// ------------------------------------------------------------------- pages
// Sums of a request's new tokens, pages asked for and pages given back.
struct Sums {
    long long grow, need, back;
};

__device__ __forceinline__ Sums operator+(Sums a, Sums b) { return {a.grow + b.grow, a.need + b.need, a.back + b.back}; }

__device__ __forceinline__ Sums warp_scan(Sums v, int lane) {
    for (int d = 1; d < 32; d <<= 1) {
        const Sums u = {__shfl_up_sync(~0u, v.grow, d), __shfl_up_sync(~0u, v.need, d), __shfl_up_sync(~0u, v.back, d)};
        if (lane >= d) v = v + u;
    }
    return v;
}

constexpr int kPagesThreads = 1024;

// Last of the n ascending values that is at most x (the first is).
__device__ __forceinline__ int last_at_most(const long long* v, int n, long long x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// A sum of new tokens as the int32 of `starts`: those past 2³¹ − 1 have no rows, and must not come out as rows of others.
__device__ __forceinline__ int row_number(long long sum) { return static_cast<int>(min(sum, 0x7fffffffll)); }

// Every CTA scans all requests' sums, one per thread at a time, and writes
// every gridDim.x-th block of tokens and of returned pages; CTA 0 writes what
// there is one of for each request.  Reading the lengths again in every CTA
// costs less than a second launch or a barrier over the grid.  Bound by its
// chain of latencies (two loads, two barriers, a search) at every size that
// fits a cache: 3.5 µs for a decode step of 64 requests, 7.0 for 1000 requests
// between verify passes, 5.3 for prompts of 37 requests.
__global__ void __launch_bounds__(kPagesThreads) kv_pages_kernel(KvPagesArgs a) {
    __shared__ long long s_start[kPagesThreads], s_back[kPagesThreads], s_first[kPagesThreads];
    __shared__ int s_len[kPagesThreads], s_have[kPagesThreads], s_want[kPagesThreads];
    __shared__ Sums s_warp[32];
    __shared__ long long s_used[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
    const long long head = a.range[0], tail = a.range[1];
    const long long most = static_cast<long long>(a.width) * a.page_size;
    // Ring places of the counters; entries beyond wrap by one subtraction.
    const long long head_at = static_cast<long long>(static_cast<uint64_t>(head) % static_cast<uint64_t>(a.pages));
    const long long tail_at = static_cast<long long>(static_cast<uint64_t>(tail) % static_cast<uint64_t>(a.pages));
    auto ring = [&](long long at, long long i) -> int* {
        i += at;
        if (i >= a.pages) i -= a.pages;
        return a.ring + (i >= 0 && i < a.pages ? i : 0);
    };
    auto page_index = [&](int token) {  // token / page_size
        return static_cast<int>((static_cast<uint64_t>(token) * a.page_mul) >> a.page_shift);
    };
    const long long free = min(max(tail - head, 0ll), static_cast<long long>(a.pages));
    Sums carry = {0, 0, 0};
    long long used = 0;

    for (int base = 0; base < a.B; base += threads) {
        const int n = min(a.B - base, threads);
        int len = 0, target = 0;
        bool valid = false;
        if (tid < n) {
            len = a.lens[base + tid];
            target = a.target[base + tid];
            valid = len >= 0 && target >= 0 && len <= most;
            if (!valid) record_status(a.status, kStatusInvalid);
        }
        const bool fits = valid && target <= most;
        const int have = valid && len > 0 ? page_index(len - 1) + 1 : 0;
        const int want = valid && target > 0 ? page_index(target - 1) + 1 : 0;
        const Sums own = {valid ? max(target - len, 0) : 0, fits ? max(want - have, 0) : 0, max(have - want, 0)};
        Sums sum = warp_scan(own, lane);
        if (lane == 31) s_warp[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            const Sums w = lane < threads / 32 ? s_warp[lane] : Sums{0, 0, 0};
            s_warp[lane] = warp_scan(w, lane);
        }
        __syncthreads();
        if (warp > 0) sum = sum + s_warp[warp - 1];
        sum = sum + carry;
        const Sums total = carry + s_warp[threads / 32 - 1];
        const bool roomy = own.grow == 0 || sum.grow <= a.T;
        if (!roomy) record_status(a.status, kStatusInvalid);
        const bool granted = fits && roomy && (own.need == 0 || sum.need <= free);
        s_start[tid] = sum.grow - own.grow;
        s_back[tid] = sum.back - own.back;
        s_first[tid] = granted ? sum.need - own.need : -1;  // the request's first new page, from the ring's head; −1: no slots
        s_len[tid] = len;
        s_have[tid] = have;
        s_want[tid] = want;
        if (blockIdx.x == 0) {
            if (tid < n) {
                a.starts[base + tid] = row_number(sum.grow - own.grow);
                a.new_lens[base + tid] = granted ? target : len;
            }
            // The sums grow, so the last granted request's sum is the most that is used.
            long long u = granted && own.need > 0 ? sum.need : 0;
            for (int d = 16; d > 0; d >>= 1) u = max(u, __shfl_xor_sync(~0u, u, d));
            if (lane == 0) s_used[warp] = u;
        }
        __syncthreads();
        if (blockIdx.x == 0 && tid == 0)
            for (int w = 0; w < threads / 32; ++w) used = max(used, s_used[w]);

        const long long step = static_cast<long long>(gridDim.x) * threads;
        const long long t_end = min(total.grow, static_cast<long long>(a.T));
        for (long long t = carry.grow + static_cast<long long>(blockIdx.x) * threads + tid; t < t_end; t += step) {
            const int i = last_at_most(s_start, n, t);
            const int pos = s_len[i] + static_cast<int>(t - s_start[i]), index = page_index(pos);
            const int place = pos - index * a.page_size;
            long long slot = -1;
            if (s_first[i] >= 0) {
                int* entry = a.table + (base + i) * a.table_stride + index;
                const int fresh = index - s_have[i];
                const int page = fresh >= 0 ? *ring(head_at, s_first[i] + fresh) : *entry;
                // The first token of a new page writes its table entry.  A
                // request that grows past its last page has one such token in
                // each new page, since its own last page is full by then.
                if (fresh >= 0 && place == 0) *entry = page;
                if (page >= 0 && page < a.pages)
                    slot = static_cast<long long>(page) * a.page_size + place;
                else
                    record_status(a.status, kStatusInvalid);
            }
            a.slots[t] = slot;
            a.positions[t] = pos;
        }
        for (long long r = carry.back + static_cast<long long>(blockIdx.x) * threads + tid; r < total.back; r += step) {
            const int i = last_at_most(s_back, n, r);
            // The table may claim more pages than the pool has; each entry of the ring is then written again.
            *ring(tail_at, r < a.pages ? r : r % a.pages) = a.table[(base + i) * a.table_stride + s_want[i] + (r - s_back[i])];
        }
        carry = total;
        __syncthreads();
    }
    for (long long t = carry.grow + static_cast<long long>(blockIdx.x) * threads + tid; t < a.T;
         t += static_cast<long long>(gridDim.x) * threads) {
        a.slots[t] = -1;
        a.positions[t] = 0;
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.starts[a.B] = row_number(carry.grow);
        a.range_out[0] = head + used;
        a.range_out[1] = tail + carry.back;
    }
}

// ------------------------------------------------------------------ append
// Axis of each frequency (rotary ≤ 256), two bits each, eight to a word.
struct Axes {
    uint16_t of[16];
};

constexpr int kManyThreads = 64, kManyTokens = 8;  // (tokens to an SM)
constexpr int kBatch = 4;  // rows that a lane has in flight

// x·c + y·s for the two values of a word, every operation rounded on its own
// (as packed pairs, products and sums came back fused).
__device__ __forceinline__ uint32_t turn_pair(uint32_t x, uint32_t y, float2 c, float2 s) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(__fadd_rn(__fmul_rn(bf16_lo(x), c.x), __fmul_rn(bf16_lo(y), s.x)),
                                                   __fadd_rn(__fmul_rn(bf16_hi(x), c.y), __fmul_rn(bf16_hi(y), s.y)));
    return *reinterpret_cast<const uint32_t*>(&v);
}

// LPR lanes work on a row, lane c of them on its values 8c..8c+7.  A CTA takes
// every gridDim.x-th token: its threads ask for the token's rows (keys,
// values, queries), fetch its cosines and sines once for all of them into
// shared memory, and turn and write the rows.  blockIdx.y shares a token's rows
// among CTAs where there are few tokens.  Bound by reading and writing each row
// once: 16001 tokens, 40 query and 8 key-value heads of 128, in 79 µs (5.9 TB/s,
// 0.89 of a copy's rate); one token in 2.6 µs.  Into a cache in 8 bits, whose rows' maxima and divisions come on top: 104
// and 3.2 µs (bytes 65).
template <int THREADS, int LPR, bool Q8>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) kv_append_kernel(const __grid_constant__ KvAppendArgs a,
                                                                           const __grid_constant__ Axes axes) {
    constexpr int kGroups = THREADS / LPR;
    __shared__ __align__(16) float s_cos[2][128], s_sin[2][128];
    const int c = threadIdx.x % LPR, group0 = blockIdx.y * kGroups, group = group0 + threadIdx.x / LPR;
    const int groups = gridDim.y * kGroups;
    const int d = a.head_dim, H = a.kv_heads, F = a.rotary / 2, half = F / 8;
    const bool live = 8 * c < d, turned = 8 * c < a.rotary;
    const int rows = 2 * H + a.q_heads;
    // Rows r of a token: keys from 0, values from H, queries from 2H, so that r · head_stride counts from there.
    const __nv_bfloat16* const k_from = a.k.data + 8 * c;
    const __nv_bfloat16* const v_from = a.v.data - H * a.v.head_stride + 8 * c;
    const __nv_bfloat16* const q_from = a.q.data - 2 * H * a.q.head_stride + 8 * c;

    for (int t = blockIdx.x, turn = 0; t < a.T; t += gridDim.x, turn ^= 1) {
        long long slot = 0, at = 0, scale_at = 0;
        bool stored = false;
        float2 C[4], S[4];
        for (int r0 = group, base = group0; base < rows; r0 += kBatch * groups, base += kBatch * groups) {
            uint4 x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = r0 + i * groups;
                x[i] = make_uint4(0, 0, 0, 0);
                if (live && r < rows) {
                    const __nv_bfloat16* src = r < H       ? k_from + t * a.k.token_stride + r * a.k.head_stride
                                               : r < 2 * H ? v_from + t * a.v.token_stride + r * a.v.head_stride
                                                           : q_from + t * a.q.token_stride + r * a.q.head_stride;
                    x[i] = *reinterpret_cast<const uint4*>(src);
                }
            }
            if (base == group0) {
                slot = a.slots[t];
                for (int i = threadIdx.x; i < F; i += THREADS) {
                    const int axis = axes.of[i >> 3] >> (2 * (i & 7)) & 3;
                    int row = a.positions[axis * a.axis_stride + t];
                    if (row < 0 || row >= a.rows) {
                        record_status(a.status, kStatusInvalid);
                        row = 0;
                    }
                    s_cos[turn][i] = a.cos[static_cast<long long>(row) * F + i];
                    s_sin[turn][i] = a.sin[static_cast<long long>(row) * F + i];
                }
                __syncthreads();
                if (turned && !a.paired) {
                    // The first half takes −sin of its partner's values, the second +sin.
                    const int first = 8 * (c < half ? c : c - half);
                    const float sign = c < half ? -1.f : 1.f;
#pragma unroll
                    for (int y = 0; y < 4; y += 2) {
                        const float4 u = *reinterpret_cast<const float4*>(&s_cos[turn][first + 2 * y]);
                        const float4 w = *reinterpret_cast<const float4*>(&s_sin[turn][first + 2 * y]);
                        C[y] = make_float2(u.x, u.y), C[y + 1] = make_float2(u.z, u.w);
                        S[y] = make_float2(sign * w.x, sign * w.y), S[y + 1] = make_float2(sign * w.z, sign * w.w);
                    }
                } else if (turned) {
                    const float4 u = *reinterpret_cast<const float4*>(&s_cos[turn][4 * c]);
                    const float4 w = *reinterpret_cast<const float4*>(&s_sin[turn][4 * c]);
                    C[0] = make_float2(u.x, u.x), C[1] = make_float2(u.y, u.y), C[2] = make_float2(u.z, u.z), C[3] = make_float2(u.w, u.w);
                    S[0] = make_float2(-w.x, w.x), S[1] = make_float2(-w.y, w.y), S[2] = make_float2(-w.z, w.z), S[3] = make_float2(-w.w, w.w);
                }
                stored = slot >= 0 && slot < a.pages * a.page_size;
                if (!stored && slot != -1) record_status(a.status, kStatusInvalid);
                if (stored) {
                    const long long page = slot <= 0x7fffffff
                                               ? static_cast<long long>((static_cast<uint64_t>(slot) * a.page_mul) >> a.page_shift)
                                               : slot / a.page_size;
                    const long long place = slot - page * a.page_size;
                    at = page * a.page_stride + place * a.cache_token_stride + 8 * c;
                    scale_at = page * H * a.page_size + place;
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (base + i * groups >= rows) break;  // the same for the whole CTA
                const int r = r0 + i * groups;
                const bool is_q = r >= 2 * H, is_v = !is_q && r >= H;
                const bool work = live && r < rows && (is_q || stored);
                uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t other[4];
                if (!a.paired) {
                    const int from = c < half ? c + half : c - half;
#pragma unroll
                    for (int y = 0; y < 4; ++y) other[y] = __shfl_sync(~0u, w[y], from & (LPR - 1), LPR);
                } else {
#pragma unroll
                    for (int y = 0; y < 4; ++y) other[y] = __byte_perm(w[y], 0, 0x1032);
                }
                if (turned && !is_v)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        w[y] = turn_pair(w[y], other[y], C[y], S[y]);
                if (Q8 && base + i * groups < 2 * H) {
                    // RTN at 8 bits over the row's LPR lanes (idle lanes hold zeros); query rows go along unused.
                    float most = 0.f;
                    bool finite = true;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        most = fmaxf(most, fmaxf(fabsf(bf16_lo(w[y])), fabsf(bf16_hi(w[y]))));
                        finite = finite && isfinite(bf16_lo(w[y])) && isfinite(bf16_hi(w[y]));
                    }
                    if (!finite) most = INFINITY;
#pragma unroll
                    for (int m = LPR / 2; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, m));
                    if (work && !is_q) {
                        const bool bad = isinf(most);
                        const __nv_bfloat16 scale = __float2bfloat16_rn(bad ? NAN : __fdiv_rn(most, 127.f));
                        const float s = __bfloat162float(scale);
                        uint32_t code[2] = {0, 0};
                        if (!bad && s > 0.f)
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const int q0 = __float2int_rn(fminf(fmaxf(rintf(__fdiv_rn(bf16_lo(w[y]), s)), -128.f), 127.f));
                                const int q1 = __float2int_rn(fminf(fmaxf(rintf(__fdiv_rn(bf16_hi(w[y]), s)), -128.f), 127.f));
                                code[y / 2] |= ((q0 & 0xFFu) | (q1 & 0xFFu) << 8) << (16 * (y & 1));
                            }
                        const int h = is_v ? r - H : r;
                        int8_t* dst = static_cast<int8_t*>(is_v ? a.v_cache : a.k_cache) + at + h * a.cache_head_stride;
                        *reinterpret_cast<uint2*>(dst) = make_uint2(code[0], code[1]);
                        if (c == 0) (is_v ? a.v_scales : a.k_scales)[scale_at + static_cast<long long>(h) * a.page_size] = scale;
                    }
                }
                if (work && (is_q || !Q8)) {
                    __nv_bfloat16* dst;
                    if (is_q)
                        dst = a.q_out.data + t * a.q_out.token_stride + (r - 2 * H) * a.q_out.head_stride + 8 * c;
                    else
                        dst = static_cast<__nv_bfloat16*>(is_v ? a.v_cache : a.k_cache) + at + (is_v ? r - H : r) * a.cache_head_stride;
                    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
    }
}

template <int THREADS, int LPR>
cudaError_t append(const KvAppendArgs& a, const Axes& axes, bool q8, int64_t tokens, int sm_count, cudaStream_t stream) {
    const int per_cta = THREADS / LPR, rows = 2 * a.kv_heads + a.q_heads;
    // Few tokens: a CTA for every THREADS / LPR rows, so that the rows of a token are in flight at once.  80 rows of 128
    // with and without: 2.5 and 3.6 µs for 1 token, 3.2 and 3.8 for 76, 5.0 and 3.9 for 152.
    const dim3 grid(static_cast<unsigned>(std::min(a.T, tokens)), a.T * 2 >= sm_count ? 1u : static_cast<unsigned>((rows + per_cta - 1) / per_cta));
    if (q8)
        kv_append_kernel<THREADS, LPR, true><<<grid, THREADS, 0, stream>>>(a, axes);
    else
        kv_append_kernel<THREADS, LPR, false><<<grid, THREADS, 0, stream>>>(a, axes);
    return cudaGetLastError();
}

template <int THREADS>
cudaError_t append_dim(const KvAppendArgs& a, const Axes& axes, bool q8, int64_t tokens, int sm_count, cudaStream_t stream) {
    if (a.head_dim <= 64) return append<THREADS, 8>(a, axes, q8, tokens, sm_count, stream);
    if (a.head_dim <= 128) return append<THREADS, 16>(a, axes, q8, tokens, sm_count, stream);
    return append<THREADS, 32>(a, axes, q8, tokens, sm_count, stream);
}

}  // namespace

cudaError_t launch_kv_pages(KvPagesArgs a, const DeviceInfo& dev, cudaStream_t stream) {
    divide_by(a.page_size, &a.page_mul, &a.page_shift);
    // Small CTAs' barriers cost less, but each thread scans one request at a time: 3.2 µs with 256 threads and 4.2 with
    // 1024 for 64 requests (a token each), 3.6 and 4.7 for 256, 5.5 and 4.8 for 384, 9.4 and 5.6 for 1000.
    const int threads = a.B <= 256 ? 256 : kPagesThreads;
    const int64_t blocks = (a.T + threads - 1) / threads;
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(blocks, dev.sm_count * (kPagesThreads / threads))));
    kv_pages_kernel<<<grid, threads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(KvAppendArgs a, const int32_t sections[4], bool cycled, bool q8, const DeviceInfo& dev,
                             cudaStream_t stream) {
    divide_by(a.page_size, &a.page_mul, &a.page_shift);
    Axes axes = {};
    int used[4] = {0, 0, 0, 0};
    for (int i = 0, turn = 0; i < a.rotary / 2; ++i) {
        while (used[turn % a.axes] == sections[turn % a.axes]) ++turn;
        const int axis = turn % a.axes;
        axes.of[i >> 3] |= static_cast<uint16_t>(axis << (2 * (i & 7)));
        ++used[axis];
        if (cycled) ++turn;
    }
    // Small CTAs wait less for one another between tokens, large ones have a token's rows in flight sooner.  56 rows
    // of 128: 208 tokens take 3.7 µs with 256 threads and 5.9 with 64, 800 take 6.6 and 7.2, 1600 14.1 and 12.4,
    // 5000 34 and 30, 16001 100 and 78 (81 with 128).
    if (a.T >= kManyTokens * dev.sm_count) return append_dim<kManyThreads>(a, axes, q8, 1024 / kManyThreads * dev.sm_count, dev.sm_count, stream);
    return append_dim<256>(a, axes, q8, 4 * dev.sm_count, dev.sm_count, stream);
}

}  // namespace w4
