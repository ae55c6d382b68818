// Attention of the newest tokens of each request over its pages of the
// key-value cache.
//
// For a row at position p: o = Σ_t exp(s_t − m) v_t / Σ_t exp(s_t − m) over the
// tokens it sees, s_t = scale · q·k_t and m the largest s_t, in one pass over
// the tokens: where the running maximum grows from m to m', sums and values so
// far are multiplied by exp(m − m').
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "w4_device.cuh"
#include "w4_kv.h"

namespace w4 {
namespace {

constexpr int kWarps = 4;

// One CTA per row and query head; its warps take the tokens in turn, a lane
// holds values lane, lane + 32, ... of the row.
template <bool Q8>
__global__ void __launch_bounds__(kWarps * 32) attn_row_kernel(AttnArgs a) {
    const long long t = blockIdx.x / a.q_heads;
    const int hq = blockIdx.x % a.q_heads, h = hq / (a.q_heads / a.kv_heads);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = a.head_dim;
    int b;
    long long first, last;  // rows of the request
    if (a.starts) {
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (a.starts[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        b = lo;
        first = a.starts[b];
        last = min(static_cast<long long>(a.starts[b + 1]), static_cast<long long>(a.T));
        if (t < first || t >= last) return;
    } else {
        const long long n = a.T / a.B;
        b = static_cast<int>(t / n);
        first = b * n;
        last = first + n;
    }
    long long len = a.lens[b];
    const long long most = static_cast<long long>(a.width) * a.page_size;
    if (len < 0 || len > most) {
        record_status(a.status, kStatusInvalid);
        len = len < 0 ? 0 : most;
    }
    const long long pos = len - (last - first) + (t - first);
    const long long begin = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;

    float q[8], o[8];
    const __nv_bfloat16* qrow = a.q.data + t * a.q.token_stride + hq * a.q.head_stride;
    for (int i = 0; i < 8; ++i) {
        q[i] = lane + 32 * i < d ? __bfloat162float(qrow[lane + 32 * i]) : 0.f;
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (long long token = begin + warp; token <= pos; token += kWarps) {
        const long long page = a.table[b * a.table_stride + token / a.page_size];
        const bool there = page >= 0 && page < a.pages;
        if (!there) record_status(a.status, kStatusInvalid);
        const long long row =
            there ? page * a.page_stride + token % a.page_size * a.token_stride + h * a.head_stride : 0;
        const long long scale_at = there && Q8 ? (page * a.kv_heads + h) * a.page_size + token % a.page_size : 0;
        auto value = [&](const void* base, const __nv_bfloat16* scales, int i) {
            if (!there || lane + 32 * i >= d) return 0.f;
            if (Q8)
                return static_cast<float>(static_cast<const int8_t*>(base)[row + lane + 32 * i]) *
                       __bfloat162float(scales[scale_at]);
            return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[row + lane + 32 * i]);
        };
        float s = 0.f;
        for (int i = 0; i < 8; ++i) s += q[i] * value(a.k, a.k_scales, i);
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
        s *= a.scale;
        const float grown = fmaxf(m, s);
        const float keep = m == -INFINITY ? 0.f : expf(m - grown), p = expf(s - grown);
        m = grown;
        l = l * keep + p;
        for (int i = 0; i < 8; ++i) o[i] = o[i] * keep + p * value(a.v, a.v_scales, i);
    }

    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][256];
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
    for (int i = 0; i < 8; ++i) s_o[warp][lane + 32 * i] = o[i];
    __syncthreads();
    __nv_bfloat16* orow = a.out.data + t * a.out.token_stride + hq * a.out.head_stride;
    for (int x = threadIdx.x; x < d; x += kWarps * 32) {
        float mm = -INFINITY, ll = 0.f, oo = 0.f;
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w]);
        for (int w = 0; w < kWarps; ++w) {
            const float f = s_m[w] == -INFINITY && s_l[w] == 0.f ? 0.f : expf(s_m[w] - mm);
            ll += f * s_l[w];
            oo += f * s_o[w][x];
        }
        orow[x] = __float2bfloat16_rn(pos < 0 ? 0.f : oo / ll);
    }
}

}  // namespace

size_t attn_decode_workspace_bytes(int32_t, int64_t, int32_t, int32_t, int32_t) { return 256; }

cudaError_t launch_attn_decode(const AttnArgs& a, bool q8, void*, const DeviceInfo&, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(a.T * a.q_heads);
    if (q8)
        attn_row_kernel<true><<<grid, kWarps * 32, 0, stream>>>(a);
    else
        attn_row_kernel<false><<<grid, kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace w4
