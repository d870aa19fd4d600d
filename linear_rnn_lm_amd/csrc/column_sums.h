// column_sums.h -- sums over the rows of a matrix of partial sums, in a fixed order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sums {

// The sums of the n columns of `part` (rows x n): the first n0 of them to out0, the next n1 to out1,
// the rest to out2.  Any output may be NULL.
hipError_t launch_column_sums(const float* part, int rows, int64_t n, float* out0, int64_t n0, float* out1, int64_t n1,
                              float* out2, hipStream_t s);

}  // namespace sums
