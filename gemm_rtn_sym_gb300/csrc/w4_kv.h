// Internal declarations of the paged key-value cache's operators (host side
// and kernel arguments).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "w4_internal.h"

namespace w4 {

struct KvPagesArgs {
    const int32_t* lens;
    const int32_t* target;
    int32_t B;
    int32_t page_size;
    int32_t* ring;
    int64_t pages;
    const int64_t* range;
    int32_t* table;
    int64_t table_stride;
    int32_t width;
    int64_t T;
    int32_t* new_lens;
    int32_t* starts;
    int64_t* slots;
    int32_t* positions;
    int64_t* range_out;
    unsigned* status;
    uint32_t page_mul;  // divide_by(page_size)
    int32_t page_shift;
};

// bf16 rows [tokens, heads, head_dim], strides in elements.
struct Rows {
    __nv_bfloat16* data;
    int64_t token_stride;
    int64_t head_stride;
};

struct KvAppendArgs {
    Rows q, q_out, k, v;
    int32_t q_heads, kv_heads, head_dim;
    int64_t T;
    const int32_t* positions;
    int64_t axis_stride;
    const float* cos;
    const float* sin;
    int64_t rows;
    int32_t rotary;
    int32_t axes;
    int32_t paired;
    void* k_cache;
    void* v_cache;
    __nv_bfloat16* k_scales;
    __nv_bfloat16* v_scales;
    int64_t pages;
    int64_t page_stride, cache_token_stride, cache_head_stride;
    int32_t page_size;
    const int64_t* slots;
    unsigned* status;
    uint32_t page_mul;  // divide_by(page_size)
    int32_t page_shift;
};

struct AttnArgs {
    Rows q, out;
    int32_t B;
    int64_t T;
    int32_t q_heads, kv_heads, head_dim;
    const void* k;
    const void* v;
    const __nv_bfloat16* k_scales;
    const __nv_bfloat16* v_scales;
    int64_t pages;
    int64_t page_stride, token_stride, head_stride;
    int32_t page_size;
    const int32_t* table;
    int64_t table_stride;
    int32_t width;
    const int32_t* lens;
    const int32_t* starts;  // nullptr: T / B rows each
    float scale;
    int64_t window;
    unsigned* status;
    uint32_t page_mul;  // divide_by(page_size)
    int32_t page_shift;
};

// n / by = (n · mul) >> shift for every n < 2³¹: mul = ⌈2^shift / by⌉ with shift
// = 31 + l and 2^l ≥ by errs by less than n / 2^(31 + l) < 1 / by, and fits 32 bits.
inline void divide_by(int32_t by, uint32_t* mul, int32_t* shift) {
    int l = 0;
    while ((int64_t{1} << l) < by) ++l;
    *shift = 31 + l;
    *mul = static_cast<uint32_t>(((uint64_t{1} << *shift) + static_cast<uint64_t>(by) - 1) / static_cast<uint64_t>(by));
}

// Arguments are already validated by the C ABI layer; the divisors are filled in here.
cudaError_t launch_kv_pages(KvPagesArgs a, const DeviceInfo& dev, cudaStream_t stream);
cudaError_t launch_kv_append(KvAppendArgs a, const int32_t sections[4], bool cycled, bool q8, const DeviceInfo& dev,
                             cudaStream_t stream);
size_t attn_decode_workspace_bytes(int32_t B, int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim, bool q8);
cudaError_t launch_attn_decode(AttnArgs a, bool q8, void* workspace, const DeviceInfo& dev,
                               cudaStream_t stream);

}  // namespace w4
