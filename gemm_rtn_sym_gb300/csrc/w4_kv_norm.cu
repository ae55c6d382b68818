// Queries and keys of new tokens normalised head by head, turned by their
// rotary positions and written to the cache, in one pass over the rows.
//
//   r = (Σ x² / head_dim + eps)^−½,  y = x · r · (w + offset),  then the turn
//   (a, b) → (a·cos − b·sin, b·cos + a·sin), all in fp32, rounded once
//
// A row is read once and written once; its sum of squares is a few shuffles
// among the lanes that hold it.  Done apart, the norm would read and write the
// queries and keys once more, and round them once more.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "w4_device.cuh"
#include "w4_kv.h"

namespace w4 {
namespace {

constexpr int kManyThreads = 64, kManyTokens = 8;  // (tokens to an SM)
constexpr int kBatch = 4;  // rows that a lane has in flight

__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// (Σ x² / n + eps)^−½ of a row whose sum in fp32 is past 10³⁷: once more with the values times the power of two that
// takes the largest near 1.  A row with an infinity keeps its sum (every finite value then becomes 0), and so does one
// with a NaN.
template <int LPR>
__device__ __forceinline__ float far_root(const float (&v)[8], float sum, const KvNorm& norm) {
    float most = 0.f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        most = fmaxf(most, fabsf(v[i]));
        finite = finite && isfinite(v[i]);
    }
    if (!finite) most = INFINITY;
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, m));
    const int e = min(max(static_cast<int>(__float_as_uint(most) >> 23), 1), 253);
    const float s = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    float scaled = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) scaled = fmaf(v[i] * s, v[i] * s, scaled);
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) scaled += __shfl_xor_sync(~0u, scaled, m);
    return isfinite(most) && !(sum < 1e37f) ? s * rsqrtf(fmaf(scaled, norm.inv_dim, norm.eps * s * s))
                                            : rsqrtf(fmaf(sum, norm.inv_dim, norm.eps));
}

// LPR lanes work on a row.  Lane c has eight of its values, in two runs of four
// that begin at columns `one` and `two`: where halves turn with one another,
// values 4c.. of the first and of the second half, so that no value has to
// come from another lane; else values 8c and 8c + 4.  A CTA takes every
// gridDim.x-th token: its threads ask for the token's rows (keys, values,
// queries), fetch its cosines and sines once for all of them, and normalise,
// turn and write.  blockIdx.y shares a token's rows among CTAs where there are
// few tokens.
template <int THREADS, int LPR, bool Q8>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) kv_append_norm_kernel(const __grid_constant__ KvAppendArgs a,
                                                                                const __grid_constant__ KvNorm norm,
                                                                                const __grid_constant__ Axes axes) {
    constexpr int kGroups = THREADS / LPR;
    __shared__ __align__(16) float s_cos[2][128], s_sin[2][128];
    const int c = threadIdx.x % LPR, group0 = blockIdx.y * kGroups, group = group0 + threadIdx.x / LPR;
    const int groups = gridDim.y * kGroups;
    const int d = a.head_dim, H = a.kv_heads, F = a.rotary / 2;
    const bool live = 8 * c < d, turned = 8 * c < a.rotary;
    const int one = turned && !a.paired ? 4 * c : 8 * c, two = turned && !a.paired ? F + 4 * c : 8 * c + 4;
    const int rows = 2 * H + a.q_heads;
    // Rows r of a token: keys from 0, values from H, queries from 2H, so that r · head_stride counts from there.
    const __nv_bfloat16* const k_from = a.k.data;
    const __nv_bfloat16* const v_from = a.v.data - H * a.v.head_stride;
    const __nv_bfloat16* const q_from = a.q.data - 2 * H * a.q.head_stride;

    float wq[8], wk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int col = (i < 4 ? one : two) + (i & 3);
        auto weight = [&](const void* w) {
            if (!live || !w) return 0.f;
            return (norm.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[col]) : static_cast<const float*>(w)[col]) + norm.offset;
        };
        wq[i] = weight(norm.q_weight);
        wk[i] = weight(norm.k_weight);
    }

    for (int t = blockIdx.x, turn = 0; t < a.T; t += gridDim.x, turn ^= 1) {
        long long slot = 0, at = 0, scale_at = 0;
        bool stored = false;
        float C[4] = {}, S[4] = {};
        for (int r0 = group, base = group0; base < rows; r0 += kBatch * groups, base += kBatch * groups) {
            uint2 x[kBatch][2];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = r0 + i * groups;
                x[i][0] = x[i][1] = make_uint2(0, 0);
                if (live && r < rows) {
                    const __nv_bfloat16* src = r < H       ? k_from + t * a.k.token_stride + r * a.k.head_stride
                                               : r < 2 * H ? v_from + t * a.v.token_stride + r * a.v.head_stride
                                                           : q_from + t * a.q.token_stride + r * a.q.head_stride;
                    x[i][0] = *reinterpret_cast<const uint2*>(src + one);
                    x[i][1] = *reinterpret_cast<const uint2*>(src + two);
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
                if (turned) {
                    const float4 u = *reinterpret_cast<const float4*>(&s_cos[turn][4 * c]);
                    const float4 w = *reinterpret_cast<const float4*>(&s_sin[turn][4 * c]);
                    C[0] = u.x, C[1] = u.y, C[2] = u.z, C[3] = u.w;
                    S[0] = w.x, S[1] = w.y, S[2] = w.z, S[3] = w.w;
                }
                stored = slot >= 0 && slot < a.pages * a.page_size;
                if (!stored && slot != -1) record_status(a.status, kStatusInvalid);
                if (stored) {
                    const long long page = slot <= 0x7fffffff
                                               ? static_cast<long long>((static_cast<uint64_t>(slot) * a.page_mul) >> a.page_shift)
                                               : slot / a.page_size;
                    const long long place = slot - page * a.page_size;
                    at = page * a.page_stride + place * a.cache_token_stride;
                    scale_at = page * H * a.page_size + place;
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (base + i * groups >= rows) break;  // the same for the whole CTA
                const int r = r0 + i * groups;
                const bool is_q = r >= 2 * H, is_v = !is_q && r >= H;
                const bool work = live && r < rows && (is_q || stored);
                float v[8] = {bf16_lo(x[i][0].x), bf16_hi(x[i][0].x), bf16_lo(x[i][0].y), bf16_hi(x[i][0].y),
                              bf16_lo(x[i][1].x), bf16_hi(x[i][1].x), bf16_lo(x[i][1].y), bf16_hi(x[i][1].y)};
                float sum = 0.f;
#pragma unroll
                for (int y = 0; y < 8; ++y) sum = fmaf(v[y], v[y], sum);
#pragma unroll
                for (int m = LPR / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(~0u, sum, m);
                float root = rsqrtf(fmaf(sum, norm.inv_dim, norm.eps));
                if (__any_sync(~0u, !(sum < 1e37f))) root = far_root<LPR>(v, sum, norm);
                if (!is_v) {
#pragma unroll
                    for (int y = 0; y < 8; ++y) v[y] *= root * (is_q ? wq[y] : wk[y]);
                    if (turned && a.paired) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float one_was = v[2 * y];
                            v[2 * y] = one_was * C[y] - v[2 * y + 1] * S[y];
                            v[2 * y + 1] = v[2 * y + 1] * C[y] + one_was * S[y];
                        }
                    } else if (turned) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float one_was = v[y];
                            v[y] = one_was * C[y] - v[y + 4] * S[y];
                            v[y + 4] = v[y + 4] * C[y] + one_was * S[y];
                        }
                    }
                }
                if (Q8 && base + i * groups < 2 * H) {
                    // RTN at 8 bits over the row's LPR lanes (idle lanes hold zeros); query rows go along unused.
                    float most = 0.f;
                    bool finite = true;
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        most = fmaxf(most, fabsf(v[y]));
                        finite = finite && isfinite(v[y]);
                    }
                    if (!finite && live) most = INFINITY;
#pragma unroll
                    for (int m = LPR / 2; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, m));
                    if (work && !is_q) {
                        const bool bad = isinf(most);
                        const __nv_bfloat16 scale = __float2bfloat16_rn(bad ? NAN : __fdiv_rn(most, 127.f));
                        const float s = __bfloat162float(scale);
                        uint32_t code[2] = {0, 0};
                        if (!bad && s > 0.f)
#pragma unroll
                            for (int y = 0; y < 8; ++y) {
                                const int q = __float2int_rn(fminf(fmaxf(rintf(__fdiv_rn(v[y], s)), -128.f), 127.f));
                                code[y / 4] |= (q & 0xFFu) << (8 * (y & 3));
                            }
                        const int h = is_v ? r - H : r;
                        int8_t* dst = static_cast<int8_t*>(is_v ? a.v_cache : a.k_cache) + at + h * a.cache_head_stride;
                        *reinterpret_cast<uint32_t*>(dst + one) = code[0];
                        *reinterpret_cast<uint32_t*>(dst + two) = code[1];
                        if (c == 0) (is_v ? a.v_scales : a.k_scales)[scale_at + static_cast<long long>(h) * a.page_size] = scale;
                    }
                }
                if (work && (is_q || !Q8)) {
                    __nv_bfloat16* dst;
                    if (is_q)
                        dst = a.q_out.data + t * a.q_out.token_stride + (r - 2 * H) * a.q_out.head_stride;
                    else
                        dst = static_cast<__nv_bfloat16*>(is_v ? a.v_cache : a.k_cache) + at + (is_v ? r - H : r) * a.cache_head_stride;
                    if (is_v) {  // (as they are, NaN's bits among them)
                        *reinterpret_cast<uint2*>(dst + one) = x[i][0];
                        *reinterpret_cast<uint2*>(dst + two) = x[i][1];
                    } else {
                        *reinterpret_cast<uint2*>(dst + one) = make_uint2(pair_bf16(v[0], v[1]), pair_bf16(v[2], v[3]));
                        *reinterpret_cast<uint2*>(dst + two) = make_uint2(pair_bf16(v[4], v[5]), pair_bf16(v[6], v[7]));
                    }
                }
            }
        }
    }
}

template <int THREADS, int LPR>
cudaError_t append(const KvAppendArgs& a, const KvNorm& norm, const Axes& axes, bool q8, int64_t tokens, int sm_count, cudaStream_t stream) {
    const int per_cta = THREADS / LPR, rows = 2 * a.kv_heads + a.q_heads;
    const dim3 grid(static_cast<unsigned>(std::min(a.T, tokens)), a.T * 2 >= sm_count ? 1u : static_cast<unsigned>((rows + per_cta - 1) / per_cta));
    if (q8)
        kv_append_norm_kernel<THREADS, LPR, true><<<grid, THREADS, 0, stream>>>(a, norm, axes);
    else
        kv_append_norm_kernel<THREADS, LPR, false><<<grid, THREADS, 0, stream>>>(a, norm, axes);
    return cudaGetLastError();
}

template <int THREADS>
cudaError_t append_dim(const KvAppendArgs& a, const KvNorm& norm, const Axes& axes, bool q8, int64_t tokens, int sm_count, cudaStream_t stream) {
    if (a.head_dim <= 64) return append<THREADS, 8>(a, norm, axes, q8, tokens, sm_count, stream);
    if (a.head_dim <= 128) return append<THREADS, 16>(a, norm, axes, q8, tokens, sm_count, stream);
    return append<THREADS, 32>(a, norm, axes, q8, tokens, sm_count, stream);
}

}  // namespace

cudaError_t launch_kv_append_norm(KvAppendArgs a, const KvNorm& norm, const int32_t sections[4], bool cycled, bool q8,
                                  const DeviceInfo& dev, cudaStream_t stream) {
    divide_by(a.page_size, &a.page_mul, &a.page_shift);
    const Axes axes = axes_of(a.rotary / 2, a.axes, sections, cycled);
    if (a.T >= kManyTokens * dev.sm_count)
        return append_dim<kManyThreads>(a, norm, axes, q8, 1024 / kManyThreads * dev.sm_count, dev.sm_count, stream);
    return append_dim<256>(a, norm, axes, q8, 4 * dev.sm_count, dev.sm_count, stream);
}

}  // namespace w4
