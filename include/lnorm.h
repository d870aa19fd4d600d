/*
 * lnorm.h -- C ABI of the layer norm in libwkv7, forward and backward, on AMD
 * Instinct MI355X (gfx950): the norm in front of a time mix, and, with groups =
 * heads, the per-head norm of its output.
 *
 * Each row of C channels is cut into `groups` equal parts of D = C / groups;
 * every part is normalised by itself:
 *
 *     y = (x - mean) * rstd * weight + bias,   rstd = 1 / sqrt(var + eps)
 *
 * with mean and var over the part's D channels and one weight and bias per
 * channel (C of each).
 *
 * Conventions (status codes, dtypes, streams, ownership and error handling are
 * those of wkv7.h)
 * - x, y, dy, dx: dense (rows, C).  x and dx are x_dtype, y and dy are y_dtype,
 *   which is x_dtype or, for fp32 x, also bf16.  weight and bias are w_dtype.
 *   mean, rstd: (rows, groups) fp32.  dweight, dbias: (C) fp32.
 * - Statistics, sums and gradients are fp32 (the variance from the centred
 *   values); y and dx are rounded once.  NaN and Inf inputs propagate within their part.
 * - groups divides C, and D is at most 16384; C is at most 2^26, groups 2^20.
 * - Every pointer is a device pointer aligned to 16 bytes (mean, rstd, dweight and
 *   dbias: 4; where D is no multiple of 8, x, y, dy, dx, weight and bias: their values').
 * - Results do not vary from run to run: the sums over the rows go through
 *   per-workgroup parts in a fixed order, without atomics.
 */
#ifndef LNORM_H
#define LNORM_H

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Forward.
 *   weight, bias : or NULL for 1 and 0.
 *   y            : output, required.   mean, rstd : outputs, or both NULL.
 */
wkv7_status ln_fwd(int64_t rows, int C, int groups, wkv7_dtype x_dtype, wkv7_dtype y_dtype, wkv7_dtype w_dtype,
                   const void *x, const void *weight, const void *bias, float eps,
                   void *y, float *mean, float *rstd, void *stream);

/* Device workspace of ln_bwd.  0 for invalid shapes. */
size_t ln_bwd_workspace_bytes(int64_t rows, int C, int groups);

/*
 * Backward, with mean and rstd from ln_fwd for the same x, groups and eps.
 *   dx, dweight, dbias : outputs; dx may be NULL, and so may dweight and dbias together.
 */
wkv7_status ln_bwd(int64_t rows, int C, int groups, wkv7_dtype x_dtype, wkv7_dtype y_dtype, wkv7_dtype w_dtype,
                   const void *dy, const void *x, const void *weight, const float *mean, const float *rstd,
                   void *dx, float *dweight, float *dbias,
                   void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LNORM_H */
