// Queries and keys of new tokens normalised head by head, turned by their
// rotary positions and written to the cache, in one pass over the rows.
//
//   r = (Σ x² / head_dim + eps)^−½,  y = x · r · (w + offset),  then the turn
//   (a, b) → (a·cos − b·sin, b·cos + a·sin), all in fp32, rounded once
//
// A row is read once and written once; its sum of squares is a few shuffles
// among the lanes that hold it.  Done apart, the norm would read and write the
// queries and keys once more, and round them once more.
//
// Measured, 40 query and 8 key-value heads of 128 in bf16: 16001 tokens 87 µs,
// 0.80 of the rate of a plain copy (78.8 without norms); 208 tokens, 64 and 8
// heads, 5.5 (4.3); one token, 16 and 4 heads of 256, 3.0 (2.6).  Long prompts
// are bound by what a row takes on the way, shuffles, products and roundings
// (issue 64 %, loads' latency 45 % of the stalls at 14 of 64 resident warps);
// few tokens by one chain of latencies.
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

__device__ __forceinline__ uint32_t pair_bf16(uint64_t x) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(first_of(x), second_of(x));
    return *reinterpret_cast<const uint32_t*>(&v);
}

// (Σ x² / n + eps)^−½ of a row whose sum in fp32 is past 10³⁷: once more with the values times the power of two that
// takes the largest near 1.  A row with an infinity keeps its sum (every finite value then becomes 0), and so does one
// with a NaN.
template <int LPR>
__device__ __forceinline__ float far_root(const uint64_t (&v)[4], float sum, const KvNorm& norm) {
    float most = 0.f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        most = fmaxf(most, fmaxf(fabsf(first_of(v[i])), fabsf(second_of(v[i]))));
        finite = finite && isfinite(first_of(v[i])) && isfinite(second_of(v[i]));
    }
    if (!finite) most = INFINITY;
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, m));
    const int e = min(max(static_cast<int>(__float_as_uint(most) >> 23), 1), 253);
    const float s = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    float scaled = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) scaled = fmaf(first_of(v[i]) * s, first_of(v[i]) * s, fmaf(second_of(v[i]) * s, second_of(v[i]) * s, scaled));
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) scaled += __shfl_xor_sync(~0u, scaled, m);
    return isfinite(most) && !(sum < 1e37f) ? s * rsqrtf(fmaf(scaled, norm.inv_dim, norm.eps * s * s))
                                            : rsqrtf(fmaf(sum, norm.inv_dim, norm.eps));
}

enum Kind { kKey, kValue, kQuery };

// What a thread knows of the rows that it works on: LPR lanes to a row.  Lane c has eight of its values, in two runs of
// four that begin at columns `one` and `other`: where halves turn with one another, values 4c.. of the first and of the
// second half, so that no value has to come from another lane; else values 8c and 8c + 4.
struct Lane {
    int one, other;
    bool live, turned, paired;
};

// The turn of a token: cosines and sines of the lane's four frequencies.
struct Turned {
    uint64_t C[2], S[2], minus[2];
};

__device__ __forceinline__ void turn_values(uint64_t (&v)[4], const Turned& t, bool paired) {
    if (paired) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {  // the two of a pair, by one cosine and sine
            const float cos = y & 1 ? second_of(t.C[y >> 1]) : first_of(t.C[y >> 1]), sin = y & 1 ? second_of(t.S[y >> 1]) : first_of(t.S[y >> 1]);
            v[y] = fma2(two(second_of(v[y]), first_of(v[y])), two(-sin, sin), mul2(v[y], two(cos, cos)));
        }
    } else {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const uint64_t was = v[y];
            v[y] = fma2(v[y + 2], t.minus[y], mul2(was, t.C[y]));
            v[y + 2] = fma2(was, t.S[y], mul2(v[y + 2], t.C[y]));
        }
    }
}

// Row's codes and scale by RTN at 8 bits of its fp32 values, over its LPR lanes (idle ones hold zeros).
template <int LPR>
__device__ __forceinline__ void put_codes(const uint64_t (&v)[4], const Lane& lane, bool store, int8_t* to, __nv_bfloat16* scale_to) {
    float most = 0.f;
    bool finite = true;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        most = fmaxf(most, fmaxf(fabsf(first_of(v[y])), fabsf(second_of(v[y]))));
        finite = finite && isfinite(first_of(v[y])) && isfinite(second_of(v[y]));
    }
    if (!finite && lane.live) most = INFINITY;
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, m));
    if (!store) return;
    const bool bad = isinf(most);
    const __nv_bfloat16 scale = __float2bfloat16_rn(bad ? NAN : __fdiv_rn(most, 127.f));
    const float s = __bfloat162float(scale);
    uint32_t code[2] = {0, 0};
    if (!bad && s > 0.f)
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const int q = __float2int_rn(fminf(fmaxf(rintf(__fdiv_rn(y & 1 ? second_of(v[y >> 1]) : first_of(v[y >> 1]), s)), -128.f), 127.f));
            code[y / 4] |= (q & 0xFFu) << (8 * (y & 3));
        }
    *reinterpret_cast<uint32_t*>(to + lane.one) = code[0];
    *reinterpret_cast<uint32_t*>(to + lane.other) = code[1];
    if (threadIdx.x % LPR == 0) *scale_to = scale;
}

// A token's rows of one kind: `rows` of them, every groups-th of which, from `group` on, is this thread's; `first` is the
// same for the whole CTA.
struct Part {
    const __nv_bfloat16* from;
    int64_t stride;
    int rows, first, group, groups;
};

// A thread's next rows of a part, all loads at once; src moves behind them.
__device__ __forceinline__ void load_rows(const Part& p, const Lane& lane, const __nv_bfloat16*& src, int r, uint2 (&x)[kBatch][2]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i, src += p.groups * p.stride) {
        x[i][0] = x[i][1] = make_uint2(0, 0);
        if (lane.live && r + i * p.groups < p.rows) {
            x[i][0] = *reinterpret_cast<const uint2*>(src + lane.one);
            x[i][1] = *reinterpret_cast<const uint2*>(src + lane.other);
        }
    }
}

// weight: fp32 [head_dim] in shared memory.  x: the first rows, where they are loaded already.
template <int KIND, int LPR, bool Q8>
__device__ __forceinline__ void put_rows(const KvNorm& norm, const Lane& lane, const Turned& turned, const float* weight, const Part& p, bool loaded,
                                         uint2 (&x)[kBatch][2], void* to, int64_t to_stride, __nv_bfloat16* scales, int64_t scale_stride) {
    constexpr bool kCodes = Q8 && KIND != kQuery;
    uint64_t w[4] = {};
    if (KIND != kValue && lane.live) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(weight + lane.one), b = *reinterpret_cast<const ulonglong2*>(weight + lane.other);
        w[0] = a.x, w[1] = a.y, w[2] = b.x, w[3] = b.y;
    }
    const int rows = p.rows, groups = p.groups;
    const __nv_bfloat16* src = p.from + p.group * p.stride;
    const int64_t to_step = groups * to_stride;
    int64_t at = p.group * to_stride;
    for (int r = p.group, base = p.first; base < rows; base += kBatch * groups) {
        if (!loaded)
            load_rows(p, lane, src, r, x);
        else
            src += kBatch * groups * p.stride;
        loaded = false;
#pragma unroll
        for (int i = 0; i < kBatch; ++i, r += groups, at += to_step) {
            if (base + i * groups >= rows) break;  // the same for the whole CTA
            const bool store = lane.live && r < rows;
            if (KIND == kValue && !kCodes) {  // (as they are, NaN's bits among them)
                if (store) {
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(to) + at + lane.one) = x[i][0];
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(to) + at + lane.other) = x[i][1];
                }
                continue;
            }
            uint64_t v[4] = {two(bf16_lo(x[i][0].x), bf16_hi(x[i][0].x)), two(bf16_lo(x[i][0].y), bf16_hi(x[i][0].y)),
                             two(bf16_lo(x[i][1].x), bf16_hi(x[i][1].x)), two(bf16_lo(x[i][1].y), bf16_hi(x[i][1].y))};
            if (KIND != kValue) {
                uint64_t squares = fma2(v[1], v[1], mul2(v[0], v[0]));
                squares = add2(squares, fma2(v[3], v[3], mul2(v[2], v[2])));
                float sum = first_of(squares) + second_of(squares);
#pragma unroll
                for (int m = LPR / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(~0u, sum, m);
                float root = rsqrtf(fmaf(sum, norm.inv_dim, norm.eps));
                if (__any_sync(~0u, !(sum < 1e37f))) root = far_root<LPR>(v, sum, norm);
                const uint64_t by = two(root, root);
#pragma unroll
                for (int y = 0; y < 4; ++y) v[y] = mul2(mul2(v[y], by), w[y]);
                if (lane.turned) turn_values(v, turned, lane.paired);
            }
            if (kCodes) {
                put_codes<LPR>(v, lane, store, static_cast<int8_t*>(to) + at, scales + r * scale_stride);
            } else if (store) {
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(to) + at + lane.one) = make_uint2(pair_bf16(v[0]), pair_bf16(v[1]));
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(to) + at + lane.other) = make_uint2(pair_bf16(v[2]), pair_bf16(v[3]));
            }
        }
    }
}

// A CTA takes every gridDim.x-th token: its threads fetch the token's cosines and
// sines once for all of its rows, and then read, normalise, turn and write
// keys, values and queries, kind by kind, so that a row takes few instructions
// beside its own (one loop over all kinds of rows took 190 to two rows of 128,
// and was bound by them: 104 µs for the prompt below).  blockIdx.y shares a
// token's rows among CTAs where there are few tokens.
template <int THREADS, int LPR, bool Q8>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) kv_append_norm_kernel(const __grid_constant__ KvAppendArgs a,
                                                                                const __grid_constant__ KvNorm norm,
                                                                                const __grid_constant__ Axes axes) {
    constexpr int kGroups = THREADS / LPR;
    __shared__ __align__(16) float s_cos[2][128], s_sin[2][128], s_weight[2][256];
    const int c = threadIdx.x % LPR, own = threadIdx.x / LPR;
    const int d = a.head_dim, H = a.kv_heads, F = a.rotary / 2;
    // All kinds' rows are this CTA's, or, where there are few tokens, some of one kind.
    auto slice = [&](const Rows& from, int rows, int y, int of) { return Part{from.data, from.head_stride, rows, y * kGroups, y * kGroups + own, of * kGroups}; };
    const bool all = gridDim.y == 1;
    const int q_slices = all ? 1 : (a.q_heads + kGroups - 1) / kGroups, kv_slices = all ? 1 : (H + kGroups - 1) / kGroups, y = blockIdx.y;
    const bool keys = all || (y >= q_slices && y < q_slices + kv_slices), values = all || y >= q_slices + kv_slices;
    const bool queries = (all || y < q_slices) && a.q_heads > 0;
    const Part q_part = slice(a.q, a.q_heads, all ? 0 : y, q_slices), k_part = slice(a.k, H, all ? 0 : y - q_slices, kv_slices),
               v_part = slice(a.v, H, all ? 0 : y - q_slices - kv_slices, kv_slices);
    Lane lane;
    lane.live = 8 * c < d;
    lane.turned = 8 * c < a.rotary;
    lane.paired = a.paired;
    lane.one = lane.turned && !a.paired ? 4 * c : 8 * c;
    lane.other = lane.turned && !a.paired ? F + 4 * c : 8 * c + 4;
    pdl_start();
    for (int i = threadIdx.x; i < 2 * d; i += THREADS) {  // (read behind the first token's barrier)
        const int which = i >= d, col = i - which * d;
        const void* const w = which ? norm.q_weight : norm.k_weight;
        s_weight[which][col] = !w ? 0.f : norm.offset + (norm.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[col]) : static_cast<const float*>(w)[col]);
    }
    for (int t = blockIdx.x, turn = 0; t < a.T; t += gridDim.x, turn ^= 1) {
        const long long slot = a.slots[t];
        Part qp = q_part, kp = k_part, vp = v_part;
        qp.from += t * a.q.token_stride, kp.from += t * a.k.token_stride, vp.from += t * a.v.token_stride;
        uint2 x[kBatch][2];  // the first rows' loads are under way while the token's turn is fetched
        {
            const Part p = queries ? qp : keys ? kp : vp;
            const __nv_bfloat16* src = p.from + p.group * p.stride;
            load_rows(p, lane, src, p.group, x);
        }
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
        Turned turned = {};
        if (lane.turned) {
            const float4 u = *reinterpret_cast<const float4*>(&s_cos[turn][4 * c]);
            const float4 w = *reinterpret_cast<const float4*>(&s_sin[turn][4 * c]);
            turned.C[0] = two(u.x, u.y), turned.C[1] = two(u.z, u.w);
            turned.S[0] = two(w.x, w.y), turned.S[1] = two(w.z, w.w);
            turned.minus[0] = two(-w.x, -w.y), turned.minus[1] = two(-w.z, -w.w);
        }
        if (queries)
            put_rows<kQuery, LPR, Q8>(norm, lane, turned, s_weight[1], qp, true, x, a.q_out.data + t * a.q_out.token_stride, a.q_out.head_stride, nullptr, 0);
        const bool stored = slot >= 0 && slot < a.pages * a.page_size;
        if (!stored && slot != -1) record_status(a.status, kStatusInvalid);
        if (!stored) continue;  // the same for the whole CTA
        const long long page = slot <= 0x7fffffff ? static_cast<long long>((static_cast<uint64_t>(slot) * a.page_mul) >> a.page_shift)
                                                  : slot / a.page_size;
        const long long place = slot - page * a.page_size, at = page * a.page_stride + place * a.cache_token_stride;
        const long long scale_at = page * H * a.page_size + place;
        constexpr int kSize = Q8 ? 1 : 2;
        if (keys)
            put_rows<kKey, LPR, Q8>(norm, lane, turned, s_weight[0], kp, !queries, x, static_cast<uint8_t*>(a.k_cache) + at * kSize, a.cache_head_stride,
                                    a.k_scales + scale_at, a.page_size);
        if (values)
            put_rows<kValue, LPR, Q8>(norm, lane, turned, nullptr, vp, !queries && !keys, x, static_cast<uint8_t*>(a.v_cache) + at * kSize, a.cache_head_stride,
                                      a.v_scales + scale_at, a.page_size);
    }
}

template <int THREADS, int LPR>
cudaError_t append(const KvAppendArgs& a, const KvNorm& norm, const Axes& axes, bool q8, int64_t tokens, int sm_count, cudaStream_t stream) {
    const int per_cta = THREADS / LPR;
    auto slices = [&](int rows) { return (rows + per_cta - 1) / per_cta; };
    // Few tokens: a CTA for every THREADS / LPR rows of a kind, as long as all of them fit the SMs at once.  A CTA for a
    // token and for a slice, in bf16: 64 and 8 heads of 128, 6 slices, 4.9 and 2.7 µs for 1 token, 5.1 and 4.1 for 100,
    // 5.1 and 5.2 for 112, 5.8 and 7.7 for 208; 40 and 8 heads, 5 slices, 4.7 and 4.0 for 120, 4.8 and 5.0 for 128; 16
    // and 4 of 256, 4 slices, 4.6 and 4.2 for 151, 5.2 and 5.7 for 208.  Into a cache in 8 bits: 64 and 8 heads 6.6 and
    // 4.8 for 100, 6.8 and 6.9 for 151; 16 and 4 of 256 6.3 and 4.9 for 151.
    const int all = slices(a.q_heads) + 2 * slices(a.kv_heads), y = a.T * 2 >= sm_count && a.T * all > tokens ? 1 : all;
    // A few CTAs may start before the kernel ahead of them ends (3.3 to 3.0 µs for one token, one call after another);
    // many would take its SMs' room (5.5 to 7.0 for 208 tokens, 87 to 91 for 16001).
    const dim3 grid(static_cast<unsigned>(std::min(a.T, tokens)), static_cast<unsigned>(y));
    return launch_pass(q8 ? kv_append_norm_kernel<THREADS, LPR, true> : kv_append_norm_kernel<THREADS, LPR, false>, grid, THREADS, 0, stream, y > 1, a, norm, axes);
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
