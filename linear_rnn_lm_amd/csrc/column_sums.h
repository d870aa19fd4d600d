// column_sums.h -- sums over the rows of a matrix of partial sums, in a fixed order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sums {

// out0[c] for c < n0, out1[c - n0] from there on: the sums of the n columns of `part`
// (rows x n).  Either output may be NULL.
hipError_t launch_column_sums(const float* part, int rows, int64_t n, float* out0, int64_t n0, float* out1,
                              hipStream_t s);

}  // namespace sums
