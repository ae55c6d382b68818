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

__device__ __forceinline__ Sums shfl_up(Sums v, int d) {
    return {__shfl_up_sync(~0u, v.grow, d), __shfl_up_sync(~0u, v.need, d), __shfl_up_sync(~0u, v.back, d)};
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

// Every CTA scans all requests' sums, 1024 at a time, and writes every
// gridDim.x-th block of 1024 tokens and of 1024 returned pages; CTA 0 writes
// what there is one of for each request.  Reading the lengths again in every
// CTA costs less than a second launch or a barrier over the grid.
__global__ void __launch_bounds__(kPagesThreads) kv_pages_kernel(KvPagesArgs a) {
    __shared__ long long s_start[kPagesThreads], s_back[kPagesThreads], s_first[kPagesThreads];
    __shared__ int s_len[kPagesThreads], s_want[kPagesThreads];
    __shared__ Sums s_warp[kPagesThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long head = a.range[0], tail = a.range[1], P = a.page_size;
    const long long most = static_cast<long long>(a.width) * P;
    Sums carry = {0, 0, 0};
    long long used = 0;

    for (int base = 0; base < a.B; base += kPagesThreads) {
        const int n = min(a.B - base, kPagesThreads);
        int len = 0, target = 0;
        bool valid = false;
        if (tid < n) {
            len = a.lens[base + tid];
            target = a.target[base + tid];
            valid = len >= 0 && target >= 0 && len <= most;
            if (!valid) record_status(a.status, kStatusInvalid);
        }
        const bool fits = valid && target <= most;
        const long long have = valid ? (len + P - 1) / P : 0, want = valid ? (target + P - 1) / P : 0;
        Sums own = {valid ? max(target - len, 0) : 0, fits ? max(want - have, 0ll) : 0, max(have - want, 0ll)};
        Sums sum = own;
        for (int d = 1; d < 32; d <<= 1) {
            const Sums v = shfl_up(sum, d);
            if (lane >= d) sum = sum + v;
        }
        if (lane == 31) s_warp[warp] = sum;
        __syncthreads();
        Sums before = carry, total = carry;
        for (int w = 0; w < kPagesThreads / 32; ++w) {
            if (w < warp) before = before + s_warp[w];
            total = total + s_warp[w];
        }
        sum = before + sum;
        const bool roomy = own.grow == 0 || sum.grow <= a.T;
        if (!roomy) record_status(a.status, kStatusInvalid);
        const bool granted = fits && roomy && (own.need == 0 || sum.need <= tail - head);
        s_start[tid] = sum.grow - own.grow;
        s_back[tid] = sum.back - own.back;
        // The ring position of the request's page 0, were all its pages new; −1: no slots.
        s_first[tid] = granted ? head + sum.need - own.need : -1;
        s_len[tid] = len;
        s_want[tid] = static_cast<int>(want);
        if (blockIdx.x == 0 && tid < n) {
            a.starts[base + tid] = static_cast<int>(sum.grow - own.grow);
            a.new_lens[base + tid] = granted ? target : len;
        }
        // The sums grow, so the last granted request's sum is the most that is used.
        long long u = granted && own.need > 0 ? sum.need : 0;
        for (int d = 16; d > 0; d >>= 1) u = max(u, __shfl_xor_sync(~0u, u, d));
        __syncthreads();
        if (lane == 0) s_warp[warp].need = u;
        __syncthreads();
        for (int w = 0; w < kPagesThreads / 32; ++w) used = max(used, s_warp[w].need);

        const long long t_end = min(total.grow, static_cast<long long>(a.T));
        for (long long t = carry.grow + static_cast<long long>(blockIdx.x) * kPagesThreads + tid; t < t_end;
             t += static_cast<long long>(gridDim.x) * kPagesThreads) {
            const int i = last_at_most(s_start, n, t);
            const long long pos = s_len[i] + (t - s_start[i]), index = pos / P, have_i = (s_len[i] + P - 1) / P;
            long long slot = -1;
            if (s_first[i] >= 0) {
                int* entry = a.table + (base + i) * a.table_stride + index;
                const int page = index >= have_i
                                     ? a.ring[static_cast<uint64_t>(s_first[i] + (index - have_i)) % a.pages]
                                     : *entry;
                // The first token of a new page writes its table entry.  A
                // request that grows past its last page has one such token in
                // each new page, since its own last page is full by then.
                if (index >= have_i && pos % P == 0) *entry = page;
                if (page >= 0 && page < a.pages)
                    slot = page * P + pos % P;
                else
                    record_status(a.status, kStatusInvalid);
            }
            a.slots[t] = slot;
            a.positions[t] = static_cast<int>(pos);
        }
        for (long long r = carry.back + static_cast<long long>(blockIdx.x) * kPagesThreads + tid; r < total.back;
             r += static_cast<long long>(gridDim.x) * kPagesThreads) {
            const int i = last_at_most(s_back, n, r);
            a.ring[static_cast<uint64_t>(tail + r) % a.pages] =
                a.table[(base + i) * a.table_stride + s_want[i] + (r - s_back[i])];
        }
        carry = total;
        __syncthreads();
    }
    for (long long t = carry.grow + static_cast<long long>(blockIdx.x) * kPagesThreads + tid; t < a.T;
         t += static_cast<long long>(gridDim.x) * kPagesThreads) {
        a.slots[t] = -1;
        a.positions[t] = 0;
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.starts[a.B] = static_cast<int>(carry.grow);
        a.range_out[0] = head + used;
        a.range_out[1] = tail + carry.back;
    }
}

// ------------------------------------------------------------------ append
struct Axes {
    uint8_t of[128];  // axis of each frequency (rotary ≤ 256)
};

// One CTA holds LPR lanes for each row it works on at a time; lane c of a row
// has its values 8c..8c+7.  blockIdx.x is the token, whose tables' values are
// read once per thread and used for every row the thread turns.
template <int LPR, bool Q8>
__global__ void __launch_bounds__(256) kv_append_kernel(KvAppendArgs a, Axes axes) {
    const long long t = blockIdx.x;
    const int c = threadIdx.x % LPR, group = blockIdx.y * (blockDim.x / LPR) + threadIdx.x / LPR;
    const int groups = gridDim.y * (blockDim.x / LPR);
    const int d = a.head_dim, H = a.kv_heads, F = a.rotary / 2, half = F / 8;
    const bool live = 8 * c < d, turned = 8 * c < a.rotary;

    float cs[8], sn[8];
    if (turned) {
        // Halves: frequencies 8c.. of the first half, the same again for the second.  Pairs: 4c..4c+3.
        const int first = a.paired ? 4 * c : 8 * (c < half ? c : c - half);
        for (int i = 0; i < (a.paired ? 4 : 8); ++i) {
            int row = a.positions[axes.of[first + i] * a.axis_stride + t];
            if (row < 0 || row >= a.rows) {
                record_status(a.status, kStatusInvalid);
                row = 0;
            }
            cs[i] = a.cos[static_cast<long long>(row) * F + first + i];
            sn[i] = a.sin[static_cast<long long>(row) * F + first + i];
        }
    }
    const long long slot = a.slots[t];
    const bool stored = slot >= 0 && slot < a.pages * a.page_size;
    if (!stored && slot != -1) record_status(a.status, kStatusInvalid);
    const long long page = stored ? slot / a.page_size : 0, place = stored ? slot % a.page_size : 0;

    // Rows in the order keys, values, queries; a warp's groups stay together for the shuffles.
    const int rows = 2 * H + a.q_heads;
    for (int r0 = group - group % (32 / LPR); r0 < rows; r0 += groups) {
        const int r = r0 + group % (32 / LPR);
        const bool is_q = r >= 2 * H, is_v = !is_q && r >= H;
        const int h = is_q ? r - 2 * H : is_v ? r - H : r;
        const bool work = live && r < rows && (is_q || stored);
        uint4 x = {0, 0, 0, 0};
        if (work) {
            const Rows& src = is_q ? a.q : is_v ? a.v : a.k;
            x = *reinterpret_cast<const uint4*>(src.data + t * src.token_stride + h * src.head_stride + 8 * c);
        }
        uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t other[4];
        if (!a.paired) {
            const int from = c < half ? c + half : c - half;
            for (int i = 0; i < 4; ++i) other[i] = __shfl_sync(~0u, w[i], from & (LPR - 1), LPR);
        }
        if (turned && !is_v) {
            for (int i = 0; i < 4; ++i) {
                const float lo = bf16_lo(w[i]), hi = bf16_hi(w[i]);
                float l, u;
                if (a.paired) {
                    l = __fsub_rn(__fmul_rn(lo, cs[i]), __fmul_rn(hi, sn[i]));
                    u = __fadd_rn(__fmul_rn(hi, cs[i]), __fmul_rn(lo, sn[i]));
                } else {
                    const float ol = __fmul_rn(bf16_lo(other[i]), sn[2 * i]);
                    const float oh = __fmul_rn(bf16_hi(other[i]), sn[2 * i + 1]);
                    l = __fmul_rn(lo, cs[2 * i]);
                    u = __fmul_rn(hi, cs[2 * i + 1]);
                    l = c < half ? __fsub_rn(l, ol) : __fadd_rn(l, ol);
                    u = c < half ? __fsub_rn(u, oh) : __fadd_rn(u, oh);
                }
                const __nv_bfloat162 v = __floats2bfloat162_rn(l, u);
                w[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
        }
        if (Q8 && !is_q) {
            // RTN at 8 bits over the row's LPR lanes (idle lanes hold zeros).
            float most = 0.f;
            bool finite = true;
            for (int i = 0; i < 4; ++i) {
                most = fmaxf(most, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
                finite = finite && isfinite(bf16_lo(w[i])) && isfinite(bf16_hi(w[i]));
            }
            if (!finite) most = INFINITY;
            for (int m = LPR / 2; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, m));
            if (work) {
                const bool bad = isinf(most);
                const __nv_bfloat16 scale = __float2bfloat16_rn(bad ? NAN : __fdiv_rn(most, 127.f));
                const float s = __bfloat162float(scale);
                uint32_t code[2] = {0, 0};
                if (!bad && s > 0.f)
                    for (int i = 0; i < 4; ++i) {
                        const int q0 = __float2int_rn(fminf(fmaxf(rintf(__fdiv_rn(bf16_lo(w[i]), s)), -128.f), 127.f));
                        const int q1 = __float2int_rn(fminf(fmaxf(rintf(__fdiv_rn(bf16_hi(w[i]), s)), -128.f), 127.f));
                        code[i / 2] |= ((q0 & 0xFFu) | (q1 & 0xFFu) << 8) << (16 * (i & 1));
                    }
                int8_t* dst = static_cast<int8_t*>(is_v ? a.v_cache : a.k_cache) + page * a.page_stride +
                              place * a.cache_token_stride + h * a.cache_head_stride + 8 * c;
                *reinterpret_cast<uint2*>(dst) = make_uint2(code[0], code[1]);
                if (c == 0)
                    (is_v ? a.v_scales : a.k_scales)[(page * H + h) * a.page_size + place] = scale;
            }
        } else if (work) {
            __nv_bfloat16* dst =
                is_q ? a.q_out.data + t * a.q_out.token_stride + h * a.q_out.head_stride
                     : static_cast<__nv_bfloat16*>(is_v ? a.v_cache : a.k_cache) + page * a.page_stride +
                           place * a.cache_token_stride + h * a.cache_head_stride;
            *reinterpret_cast<uint4*>(dst + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

template <int LPR>
cudaError_t append(const KvAppendArgs& a, const Axes& axes, bool q8, dim3 grid, cudaStream_t stream) {
    if (q8)
        kv_append_kernel<LPR, true><<<grid, 256, 0, stream>>>(a, axes);
    else
        kv_append_kernel<LPR, false><<<grid, 256, 0, stream>>>(a, axes);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_pages(const KvPagesArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
    const int64_t blocks = (a.T + kPagesThreads - 1) / kPagesThreads;
    const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(blocks, dev.sm_count)));
    kv_pages_kernel<<<grid, kPagesThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(const KvAppendArgs& a, const int32_t sections[4], int32_t n_axes, bool cycled, bool q8,
                             const DeviceInfo& dev, cudaStream_t stream) {
    Axes axes = {};
    int used[4] = {0, 0, 0, 0};
    for (int i = 0, turn = 0; i < a.rotary / 2; ++i) {
        if (cycled) {
            while (used[turn % n_axes] == sections[turn % n_axes]) ++turn;
        } else {
            while (used[turn] == sections[turn]) ++turn;
        }
        axes.of[i] = static_cast<uint8_t>(turn % n_axes);
        ++used[axes.of[i]];
        if (cycled) ++turn;
    }
    const int lpr = a.head_dim <= 64 ? 8 : a.head_dim <= 128 ? 16 : 32;
    const int per_cta = 256 / lpr, rows = 2 * a.kv_heads + a.q_heads;
    // Few tokens: one CTA per 256/LPR rows, so that every SM has some.
    const int split = a.T * 2 >= dev.sm_count ? 1 : (rows + per_cta - 1) / per_cta;
    const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>(split));
    if (lpr == 8) return append<8>(a, axes, q8, grid, stream);
    if (lpr == 16) return append<16>(a, axes, q8, grid, stream);
    return append<32>(a, axes, q8, grid, stream);
}

}  // namespace w4
