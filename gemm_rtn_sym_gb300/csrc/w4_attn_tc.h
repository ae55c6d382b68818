// The tensor-core kernel of attention over the paged cache, for many rows to a
// key-value head.
#pragma once

#include <cstddef>

#include "w4_attn_common.cuh"
#include "w4_internal.h"

namespace w4 {

// Floats of a part of a shared item.
size_t attn_tc_partial_floats(int head_dim);
cudaError_t launch_attn_tc(const SplitArgs& sp, bool q8, const DeviceInfo& dev, cudaStream_t stream);

}  // namespace w4
