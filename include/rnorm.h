/*
 * rnorm.h -- C ABI of the fused end of a block in libwkv7, forward and backward, on AMD
 * Instinct MI355X (gfx950): the norm of a time mix's output, its gate, the scaled residual
 * and the next block's norm, in one pass over the rows.
 *
 *     r = res + scale * act(gate) * (norm1(o) * weight + bias)
 *     h = norm2(r) * weight2 + bias2
 *
 * norm1 works on each of `groups` equal parts of a row's C channels, norm2 on the whole
 * row.  Either is a layer norm, (v - mean) / sqrt(var + eps), a root-mean-square norm,
 * v / sqrt(mean(v^2) + eps), or, norm2, left out (then there is no h).
 *
 * Conventions (status codes, dtypes, streams, ownership and error handling are
 * those of wkv7.h)
 * - Rows of C values, dense but for gate, whose rows are gate_ld values apart.  o and do are
 *   o_dtype, gate, h and their gradients io_dtype, res, r and their gradients r_dtype (io_dtype
 *   or fp32; without res: io_dtype).  o_dtype is io_dtype or fp32.  weight, bias, scale,
 *   weight2 and bias2: (C) w_dtype.  Their gradients are fp32.
 * - C is at most 8192.  With groups > 1 a part has 64, 128, 256 or 512 channels.
 * - stats: (rows, 2 groups + 2) fp32: the parts' means, their 1 / sqrt(...), then norm2's
 *   two (a mean of 0 for a root-mean-square norm).
 * - h is the norm of r before its rounding.  Statistics and sums are fp32 (variances from
 *   centred values); outputs are rounded once.  NaN and Inf propagate within their part, and
 *   through norm2 within their row.
 * - Every pointer is a device pointer.  Where C is a multiple of 8, rows and weights are
 *   aligned to 16 bytes (each of gate's rows too), else to their values.
 * - Results do not vary from run to run: sums over the rows go through per-workgroup parts
 *   in a fixed order, without atomics.
 */
#ifndef RNORM_H
#define RNORM_H

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { RN_NONE = 0, RN_LAYER = 1, RN_RMS = 2 } rn_norm;
typedef enum { RN_ONE = 0, RN_SILU = 1, RN_SIGMOID = 2 } rn_act;

/*
 * Forward.
 *   gate, res, weight, bias, scale, weight2, bias2 : or NULL (no gate, 0, 1, 0, 1, 1, 0);
 *       gate if and only if act is not RN_ONE.
 *   r     : output, required.   h : output, required if and only if norm2 is not RN_NONE.
 *   stats : output, or NULL.
 */
wkv7_status rn_fwd(int64_t rows, int C, int groups, rn_norm norm, rn_norm norm2, rn_act act, wkv7_dtype o_dtype,
                   wkv7_dtype io_dtype, wkv7_dtype r_dtype, wkv7_dtype w_dtype, float eps, float eps2,
                   const void *o, const void *gate, int64_t gate_ld, const void *res, const void *weight,
                   const void *bias, const void *scale, const void *weight2, const void *bias2,
                   void *r, void *h, float *stats, void *stream);

/* Device workspace of rn_bwd.  0 for invalid shapes. */
size_t rn_bwd_workspace_bytes(int64_t rows, int C, int groups);

/*
 * Backward, with stats from rn_fwd for the same arguments.
 *   dr, dh : gradients of r and h; either may be NULL for zero, not both (dh NULL without norm2).
 *   do_, dgate, dres : outputs; dgate is required with a gate (dense), the others may be NULL.
 *   dw     : (5, C) fp32: the gradients of weight, bias, scale, weight2 and bias2; or NULL.
 */
wkv7_status rn_bwd(int64_t rows, int C, int groups, rn_norm norm, rn_norm norm2, rn_act act, wkv7_dtype o_dtype,
                   wkv7_dtype io_dtype, wkv7_dtype r_dtype, wkv7_dtype w_dtype,
                   const void *dr, const void *dh, const void *o, const void *gate, int64_t gate_ld, const void *res,
                   const float *stats, const void *weight, const void *bias, const void *scale, const void *weight2,
                   void *do_, void *dgate, void *dres, float *dw,
                   void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* RNORM_H */
