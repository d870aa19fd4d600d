/*
 * ssm.h -- C ABI of the selective state space scan in libwkv7: a linear-RNN time
 * mix whose decay differs per channel, state and token, over whole sequences
 * (forward and backward) and token by token, on AMD Instinct MI355X (gfx950).
 *
 * Every channel carries S fp32 states h.  Per token, with input x, raw step dt,
 * vectors b and c (S each, shared by the channels of a group) and gate z:
 *
 *     delta = softplus(dt + dt_bias)          (softplus = 0: dt + dt_bias)
 *     h[s]  = exp(delta A[s]) h[s] + delta x b[s]
 *     y     = (sum_s c[s] h[s] + D x) * z sigmoid(z)
 *
 * Conventions (status codes, dtypes, streams, ownership and error handling are
 * those of wkv7.h)
 * ----------------------------------------------------------------------------
 * - S is 16, 32 or 64.  G groups share b and c: channel k reads group k / (C / G); with
 *   G > 1, C / G is a multiple of 64.
 * - Token tensors are rows of `in_dtype`: token t of batch row r is row r * T + t.  x, dt,
 *   z, y and their gradients have C values per row, b and c G * S ([g][s]).  y and the
 *   gradients are dense; each input has a distance between its rows, *_ld, in values, so
 *   that it may be a slice of a wider projection (at most 2^24; ssm_step takes any).  y and the token
 *   gradients are rounded once, at the end.  A: (C, S) fp32, D, dt_bias: (C) fp32, states: (N, C, S) fp32.
 * - Sequences.  cu_seqlens NULL: N = B sequences of T tokens.  Otherwise B must be 1 and
 *   cu_seqlens is a device array of N + 1 non-decreasing offsets in 0 .. T: sequence n is
 *   the tokens cu_seqlens[n] .. cu_seqlens[n+1] - 1, and may be empty (its final state is
 *   its initial one).  Offsets are not checked on the host; offsets out of range or
 *   decreasing give unspecified results, but no access outside the tensors.  Tokens outside
 *   every sequence are not read; their rows of y and of the token gradients stay as they were, or
 *   are set to zero with zero_outside.
 * - delta A should be at most 0; the states grow without bound otherwise.  A delta of 0
 *   passes the state on as it is, also where A is -infinity.  A NaN or Inf in x, dt or z spoils its channel of its
 *   sequence only, from its token on, in b or c every channel of the group; in the
 *   gradients what the formula lets it reach.
 * - Arithmetic, states and sums are fp32; sums of steps over a stretch of tokens 64 bits, of
 *   sums of up to four neighbours in 32.  Steps and gates are good to 8 * 2^-24 of themselves, a gate
 *   of bf16 rows to 2^-17.
 * - Checkpoints: the state entering every 16th token of a sequence.  A call has
 *   ssm_slots(...) of them: N * ceil(T / 16) dense, T / 16 + N packed.
 * - Every pointer is a device pointer aligned to its values (states, checkpoints and A: 16
 *   bytes; workspace: 16).
 * - Results do not vary from run to run.
 */
#ifndef SSM_H
#define SSM_H

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Checkpoint slots of a call (packed != 0: cu_seqlens given, N sequences; else N is
 * ignored).  0 for invalid sizes. */
int64_t ssm_slots(int B, int T, int N, int packed);

/* Bytes of what ssm_fwd leaves for ssm_bwd: slots * C * S fp32.  0 for invalid shapes. */
size_t ssm_ckpt_bytes(int B, int T, int C, int S, int G, int N, int packed);

/* Device workspaces.  0 for invalid shapes. */
size_t ssm_fwd_workspace_bytes(int B, int T, int C, int S, int G, int N, int packed);
size_t ssm_bwd_workspace_bytes(int B, int T, int C, int S, int G, int N, int packed);

/*
 * Forward over whole sequences.
 *   D, z, dt_bias : or NULL for 0, no gate and 0.
 *   h0   : initial states, or NULL for zero.
 *   y    : output, or NULL.   hT : final states, or NULL; may be h0 itself.
 *   ckpt : what ssm_bwd needs (ssm_ckpt_bytes), or NULL.
 *   At least one of y, hT, ckpt must be given.
 */
wkv7_status ssm_fwd(int B, int T, int C, int S, int G, wkv7_dtype in_dtype,
                    const void *x, int64_t x_ld, const void *dt, int64_t dt_ld, const float *A,
                    const void *b, int64_t b_ld, const void *c, int64_t c_ld, const float *D,
                    const void *z, int64_t z_ld, const float *dt_bias, int softplus,
                    const int32_t *cu_seqlens, int N, int zero_outside, const float *h0, void *y, float *ckpt, float *hT,
                    void *workspace, size_t workspace_bytes, void *stream);

/*
 * Backward.
 *   dy   : gradient of y, required, dense.   dhT : gradient of hT, or NULL for zero.
 *   ckpt : left by ssm_fwd for the same inputs, offsets and h0.
 *   dx, ddt, dA, db, dc : outputs, required.  dD, dz : outputs, required where D and z are
 *   given, else NULL.  ddt_bias : output or NULL.  dh0 : output or NULL.
 *   dA, dD and ddt_bias are sums over all tokens; db and dc over the channels of a group.
 */
wkv7_status ssm_bwd(int B, int T, int C, int S, int G, wkv7_dtype in_dtype,
                    const void *dy, const float *dhT,
                    const void *x, int64_t x_ld, const void *dt, int64_t dt_ld, const float *A,
                    const void *b, int64_t b_ld, const void *c, int64_t c_ld, const float *D,
                    const void *z, int64_t z_ld, const float *dt_bias, int softplus,
                    const int32_t *cu_seqlens, int N, int zero_outside, const float *ckpt,
                    void *dx, void *ddt, float *dA, void *db, void *dc, float *dD, void *dz, float *ddt_bias,
                    float *dh0, void *workspace, size_t workspace_bytes, void *stream);

/*
 * One or a few new tokens per sequence: B rows of T tokens, token by token, with the
 * states read and written once.
 *   state     : (P, C, S) pool, required.
 *   state_out : the updated states, required: `state` itself (in place), or another pool
 *               of the same size, of which only the states that the call works on are
 *               written.
 *   slots     : device array of B pool indices, or NULL (row r uses state r, P >= B).  A
 *               row whose slot lies outside 0 .. P - 1 has no state: its y is 0 (a padded
 *               batch) and its inputs are not read.  Rows with the same slot are
 *               consecutive tokens of one sequence, in the order of the rows.
 */
wkv7_status ssm_step(int B, int T, int C, int S, int G, wkv7_dtype in_dtype,
                     const void *x, int64_t x_ld, const void *dt, int64_t dt_ld, const float *A,
                     const void *b, int64_t b_ld, const void *c, int64_t c_ld, const float *D,
                     const void *z, int64_t z_ld, const float *dt_bias, int softplus,
                     const int32_t *slots, int P, const float *state, float *state_out, void *y, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_H */
