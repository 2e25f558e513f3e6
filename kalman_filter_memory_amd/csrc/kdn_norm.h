// kdn_norm.h -- what other operators use of the norm's kernels (host side, internal).
#pragma once

#include <hip/hip_runtime.h>

namespace kdn {

// out[d] = the sum of n rows of d floats, in a fixed order (d a multiple of 4)
hipError_t launch_column_sums(int n, int d, const float* rows, float* out, hipStream_t st);

}  // namespace kdn
