/*
 * gdr.h -- C ABI of the gated delta rule in libwkv7: a linear-RNN time mix with
 * one decay per head and token, chunked (prompts, training) and recurrent
 * (new tokens), forward and backward, on AMD Instinct MI355X (gfx950).
 *
 * Every value head carries a V x K fp32 state S, rows i paired with v and o,
 * columns j paired with q and k.  Per token t, with log decay g and write
 * strength beta:
 *
 *     S[i][j] = exp(g_t) S[i][j]
 *     u[i]    = beta_t (v_t[i] - sum_j S[i][j] k_t[j])
 *     S[i][j] = S[i][j] + u[i] k_t[j]
 *     o_t[i]  = scale sum_j S[i][j] q_t[j]
 *
 * Conventions (status codes, dtypes, streams, ownership and error handling are
 * those of wkv7.h)
 * ----------------------------------------------------------------------------
 * - K and V are 64 or 128 each.  H value heads share Hk query/key heads: H is a
 *   multiple of Hk, and value head h reads head h / (H / Hk) of q and k.
 * - q, k: dense (B, T, Hk, K); v, o, dout, dv: (B, T, H, V); all `in_dtype`.
 *   o, dq, dk and dv are rounded to in_dtype once, at the end.  g, beta, dg,
 *   dbeta: (B, T, H) fp32.  States: (N, H, V, K) fp32 with S[i][j] at i*K + j.
 * - Sequences.  cu_seqlens NULL: N = B sequences of T tokens.  Otherwise B must
 *   be 1 and cu_seqlens is a device array of N + 1 non-decreasing offsets in
 *   0 .. T: sequence n is the tokens cu_seqlens[n] .. cu_seqlens[n+1] - 1, and
 *   may be empty (its final state is its initial one).  The offsets are not
 *   checked on the host (that would wait for the GPU); offsets out of range or
 *   decreasing give unspecified results, but no access outside the tensors.
 *   Tokens outside every sequence are neither read nor written: their rows of
 *   o, dq, dk, dv, dg and dbeta stay as they were.
 * - |k| should be at most about 1 with beta in [0, 1] (or beta |k|^2 <= 2): outside,
 *   the rule itself diverges.  g <= 0; g = -inf (any value below -200) clears the state.
 *   A beta of magnitude below 2^-60 is taken as 2^-60.
 *   A NaN or Inf input spoils its own sequence from its chunk of 64 tokens on
 *   (in the backward, up to that chunk as well), never another sequence.
 * - Arithmetic is fp32 or better throughout: products on the matrix cores use
 *   three bf16 planes per fp32 value (24 bits), sums of log decays 64 bits.
 * - Chunks are 64 tokens, counted from each sequence's first.  A call has
 *   gdr_slots(...) chunk slots: N * ceil(T / 64) dense, T / 64 + N packed.  Chunk
 *   slots times H must stay below 2^22 - 15, and N * H at most 2^20 (gdr_step: B * H
 *   below 2^22).
 * - Every pointer is a device pointer aligned to 16 bytes (g, beta, dg, dbeta,
 *   cu_seqlens, slots and what gdr_zero_outside clears: 4).
 * - Results do not vary from run to run.
 */
#ifndef GDR_H
#define GDR_H

#include "wkv7.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Chunk slots of a call (packed != 0: cu_seqlens given, N sequences; else N is
 * ignored).  0 for invalid sizes. */
int64_t gdr_slots(int B, int T, int N, int packed);

/* Bytes of what gdr_fwd leaves for gdr_bwd: slots * H blocks of
 * (K + 64) * V + 6464 fp32, per chunk and head the state entering the chunk
 * (V x K), the chunk's u (V x 64), and in a library-internal format its two
 * triangular matrices and its gates.  0 for invalid shapes. */
size_t gdr_ckpt_bytes(int B, int T, int Hk, int H, int K, int V, int N, int packed);

/* Device workspace of gdr_fwd (without and with ckpt: that holds the larger part by
 * itself) and of gdr_bwd.  0 for invalid shapes. */
size_t gdr_fwd_workspace_bytes(int B, int T, int Hk, int H, int K, int V, wkv7_dtype in_dtype, int N, int packed);
size_t gdr_fwd_train_workspace_bytes(int B, int T, int Hk, int H, int K, int V, wkv7_dtype in_dtype, int N, int packed);
size_t gdr_bwd_workspace_bytes(int B, int T, int Hk, int H, int K, int V, wkv7_dtype in_dtype, int N, int packed);

/*
 * Forward over whole sequences.
 *   h0   : initial states, or NULL for zero.
 *   o    : output, or NULL.   hT : final states, or NULL; may be h0 itself.
 *   ckpt : what gdr_bwd needs (gdr_ckpt_bytes), or NULL.
 *   At least one of o, hT, ckpt must be given.
 *   workspace: gdr_fwd_workspace_bytes bytes, with ckpt gdr_fwd_train_workspace_bytes
 *   (never more), clobbered; nothing in it is kept.
 */
wkv7_status gdr_fwd(int B, int T, int Hk, int H, int K, int V, wkv7_dtype in_dtype,
                    const void *q, const void *k, const void *v, const float *g, const float *beta,
                    const int32_t *cu_seqlens, int N, float scale,
                    const float *h0, void *o, float *ckpt, float *hT,
                    void *workspace, size_t workspace_bytes, void *stream);

/*
 * Backward.
 *   dout : gradient of o, required.   dhT : gradient of hT, or NULL for zero.
 *   ckpt : left by gdr_fwd for the same inputs, offsets and h0.
 *   dq, dk, dv, dg, dbeta : outputs, required.   dh0 : output, or NULL.
 *   Gradients of q and k are summed over the value heads that share them.
 */
wkv7_status gdr_bwd(int B, int T, int Hk, int H, int K, int V, wkv7_dtype in_dtype,
                    const void *dout, const float *dhT,
                    const void *q, const void *k, const void *v, const float *g, const float *beta,
                    const int32_t *cu_seqlens, int N, float scale, const float *ckpt,
                    void *dq, void *dk, void *dv, float *dg, float *dbeta, float *dh0,
                    void *workspace, size_t workspace_bytes, void *stream);

/*
 * Zero the rows of n token tensors (at most 8) that belong to no sequence: the
 * rows before cu_seqlens[0] and from cu_seqlens[N] on.  gdr_fwd and gdr_bwd leave
 * them as they were; a caller that hands out fresh buffers clears them with this.
 *   ptrs, row_bytes : host arrays of n device pointers and their bytes per token
 *                     (multiples of 4).
 */
wkv7_status gdr_zero_outside(int T, int N, const int32_t *cu_seqlens, int n, void *const *ptrs,
                             const int64_t *row_bytes, void *stream);

/*
 * One or a few new tokens per sequence: B rows of T tokens, evaluated token by
 * token with the states read and written once.
 *   state     : (P, H, V, K) pool, required.
 *   state_out : the updated states, required: `state` itself (in place), or
 *               another pool of the same size, of which only the states that
 *               the call works on are written.
 *   slots     : device array of B pool indices, or NULL (row b uses state b,
 *               P >= B).  A row whose slot lies outside 0 .. P - 1 has no
 *               state: its o is 0 (a padded batch).  Rows with the same slot are
 *               consecutive tokens of one sequence, in the order of the rows.
 */
wkv7_status gdr_step(int B, int T, int Hk, int H, int K, int V, wkv7_dtype in_dtype,
                     const void *q, const void *k, const void *v, const float *g, const float *beta,
                     const int32_t *slots, int P, float scale,
                     const float *state, float *state_out, void *o, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H */
