// The tensor-core kernel of attention over the paged cache, for many rows to a
// key-value head.
#pragma once

#include <cstddef>

#include "w4_attn_common.cuh"
#include "w4_internal.h"

namespace w4 {

// Floats of a part of a shared item.
size_t attn_tc_partial_floats(int head_dim);
// The rows' sums of the two passes of a call with shared prefixes.
struct JoinArgs {
    Rows out;
    int32_t B, T, q_heads, head_dim;
    const int32_t* starts;
    const float4* own;     // [T · q_heads]
    const float4* prefix;
    const float* own_values;  // [T · q_heads, head_dim]
    const float* prefix_values;
    const float* partial;  // parts of the prefixes' items
    int32_t pieces;        // that may have left parts
    int32_t D;             // their columns
    size_t part_floats;
};
cudaError_t launch_attn_join(JoinArgs a, cudaStream_t stream);
// kPrefixes for head_dim up to 128.  Like the other kernel in that pass, it leaves the parts of shared items for the join.
cudaError_t launch_attn_prefix(const SplitArgs& sp, bool q8, const DeviceInfo& dev, cudaStream_t stream);
// pass: one of a call with shared prefixes.
cudaError_t launch_attn_tc(const SplitArgs& sp, bool pass, bool q8, const DeviceInfo& dev, cudaStream_t stream);

}  // namespace w4
