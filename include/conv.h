/*
 * conv.h -- C ABI of the short causal convolution in libwkv7, one filter per channel,
 * over whole sequences (forward and backward) and token by token, on AMD Instinct MI355X
 * (gfx950): what stands in front of a time mix.
 *
 *     s_t = bias + sum_{j < W} weight[j] x_{t - W + 1 + j},   y_t = silu ? s_t sigmoid(s_t) : s_t
 *
 * with, before a sequence's first token, its state: its last W - 1 inputs, oldest first.
 *
 * Conventions (status codes, dtypes, streams, ownership and error handling are
 * those of wkv7.h; sequences are those of ssm.h)
 * - W is 2, 3 or 4.  x, y, dy, dx: rows of C values of x_dtype, token t of batch row r
 *   being row r * T + t; x has a distance x_ld between its rows, in values, the others are
 *   dense.  weight: (C, W), bias: (C), both w_dtype.  dweight, dbias: fp32.
 *   States h0, hT and their gradients: (N, W - 1, C) x_dtype.
 * - Sums are fp32; y, dx and dh0 are rounded once.  A NaN or Inf input spoils its channel of
 *   the W tokens that read it.
 * - Every pointer is a device pointer aligned to its values (workspace: 16).
 * - Results do not vary from run to run.
 */
#ifndef CONV_H
#define CONV_H

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Forward.
 *   bias, h0 : or NULL for zero.   y : output, required.   hT : output, or NULL; not h0.
 */
wkv7_status conv_fwd(int B, int T, int C, int W, wkv7_dtype x_dtype, wkv7_dtype w_dtype,
                     const void *x, int64_t x_ld, const void *weight, const void *bias, int silu,
                     const int32_t *cu_seqlens, int N, int zero_outside, const void *h0,
                     void *y, void *hT, void *stream);

/* Device workspace of conv_bwd.  0 for invalid shapes. */
size_t conv_bwd_workspace_bytes(int B, int T, int C, int W, int N, int packed);

/*
 * Backward.
 *   dhT : gradient of hT, or NULL for zero.   dx, dweight : outputs, required.
 *   dbias, dh0 : outputs, or NULL.
 */
wkv7_status conv_bwd(int B, int T, int C, int W, wkv7_dtype x_dtype, wkv7_dtype w_dtype,
                     const void *dy, const void *dhT, const void *x, int64_t x_ld, const void *weight,
                     const void *bias, int silu, const int32_t *cu_seqlens, int N, int zero_outside, const void *h0,
                     void *dx, float *dweight, float *dbias, void *dh0,
                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * One or a few new tokens per sequence: B rows of T tokens.  state, state_out: (P, W - 1, C)
 * pools, slots, padding and rows of the same slot as in ssm_step.
 */
wkv7_status conv_step(int B, int T, int C, int W, wkv7_dtype x_dtype, wkv7_dtype w_dtype,
                      const void *x, int64_t x_ld, const void *weight, const void *bias, int silu,
                      const int32_t *slots, int P, const void *state, void *state_out, void *y, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CONV_H */
