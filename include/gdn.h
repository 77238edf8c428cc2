/*
 * gdn.h -- C ABI of libkda_fwd: the gated delta rule with one decay per token and value head,
 * on one AMD Instinct MI355X (gfx950).
 *
 * The operation: for every sequence s and value head j, with q/k head h = j / (HV / H) and a
 * state S in R^{K x V} that starts at initial_state[s, j] (or zero), each token t does
 *
 *     S <- exp(g[t, j]) S;   r = v[t, j, :] - S^T k[t, h, :];
 *     S <- S + beta[t, j] k[t, h, :] r^T;   o[t, j, :] = scale * S^T q[t, h, :]
 *
 * and final_state[s, j] is S after the last token. It is kda_fwd's operation with the decay of
 * a token shared by all key dims (a KDA call with g repeated K times gives the same result).
 *
 * Conventions are kda_fwd.h's: device pointers, caller-owned, contiguous, 16-byte aligned;
 * nothing is allocated, nothing synchronises, no atomics, errors only through the return value;
 * concurrent calls use distinct workspaces and outputs. q, k and v must be finite: a NaN or an
 * infinity makes the outputs of its sequence and heads undefined from its 64-token chunk on (in
 * the backward, for the whole sequence); other sequences and heads never see it.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#include "kda_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    /* Shapes as in kda_fwd_args: a dense batch has N == B sequences of T tokens; with
       cu_seqlens B == 1 and sequence s spans [cu_seqlens[s], cu_seqlens[s + 1]).           */
    int32_t B, T, N;
    int32_t H, HV;            /* q/k heads and value heads, HV % H == 0                      */
    int32_t K, V;             /* head dims, each in {64, 128}                                */
    int32_t io;               /* kda_dtype of q, k, v, g, beta, o (and of the gradients)     */
    const void *q;            /* [B, T, H, K]                                                */
    const void *k;            /* [B, T, H, K]                                                */
    const void *v;            /* [B, T, HV, V]                                               */
    const void *g;            /* [B, T, HV]     log decay; any g <= 0 is exact to rounding,
                                 -inf included (it clears the state)                         */
    const void *beta;         /* [B, T, HV]                                                  */
    float scale;              /* output scale; <= 0 or NaN selects K^-0.5                    */
    const int64_t *cu_seqlens;/* device [N + 1] or NULL; contents as in kda_fwd_args         */
    const float *initial_state; /* [N, HV, K, V] fp32, or NULL for zeros                     */
    void *o;                  /* [B, T, HV, V]                                               */
    float *final_state;       /* [N, HV, K, V] fp32, or NULL to skip; may be the same buffer
                                 as initial_state                                            */
    /* Pre-stage (all zero: inputs used as given), as in kda_fwd_args with one gate input a
       token and value head:
         qk_l2norm     q, k rows divided by sqrt(sum of squares + 1e-6)
         beta_sigmoid  beta <- 1 / (1 + exp(-beta))
         gate          with x = g[t, j] + dt_bias[j]: KDA_GATE_SOFTPLUS
                       g <- -exp(A_log[j]) log(1 + exp(x)); KDA_GATE_BOUNDED
                       g <- lower_bound / (1 + exp(-exp(A_log[j]) x))                        */
    int32_t qk_l2norm, beta_sigmoid, gate;
    float gate_lower_bound;   /* KDA_GATE_BOUNDED: finite and < 0                            */
    const float *A_log;       /* [HV] fp32; required for a gate                              */
    const float *dt_bias;     /* [HV] fp32, or NULL for zeros                                */
} gdn_args;

/* Bytes of device workspace gdn_fwd needs (only shapes, io and whether cu_seqlens is there are
   read, and the current device's compute-unit count); 0 for arguments gdn_fwd would reject and
   for a dense batch of at most 16 tokens a sequence, which needs none. */
size_t gdn_fwd_workspace_bytes(const gdn_args *args);

/* Enqueue the forward on `stream`: 64-token chunks (a prepare kernel, then the pass over each
   sequence's chunks, split into segments where the batch is too small to fill the device), or,
   for a dense batch of at most 16 tokens a sequence, the recurrence itself. Products take bf16
   operands in parts: two for bf16 io (the states and o carry about 17 bits before their own
   rounding), three for fp32 io (24 bits). For final states to fp32 accuracy from bf16 values pass
   them as fp32. Tokens behind the last sequence are left as they were.
   The chunked form takes less than 2^28 tokens, 2^21 (sequence, value head) pairs and, with fp32
   io, 2^26 (token, value head) pairs a call; so does gdn_bwd, for any length. */
kda_status gdn_fwd(const gdn_args *args, void *workspace, size_t ws_bytes, void *stream);

/* Gradients of gdn_fwd's inputs from the gradients of a loss with respect to o (d_o, like o) and to
   final_state (dht, fp32 [N, HV, K, V], or NULL for zero). args as for gdn_fwd (raw inputs with
   the pre-stage on; o and final_state are not read). Written, caller-owned, 16-byte aligned:
     dq, dk, dv, dg, dbeta   shapes and io dtype of q, k, v, g, beta; dq, dk summed over the value
                             heads of a q/k head, dq, dk, dg, dbeta those of the raw inputs
     dh0                     [N, HV, K, V] fp32, or NULL to skip
     dA_log, ddt_bias        [HV] fp32 (4-byte aligned): with a gate, dA_log required, ddt_bias or
                             NULL; ignored without
   bf16 io: the states and their gradients travel in two bf16 parts as in gdn_fwd (dh0 carries
   about 17 bits); for the other gradients the states, their gradients, e, v's gradient and d_o enter
   with 11 bits (fp16 with a power of two for each state, and for each token's row of the others; what
   lies 2^-28 and more below the largest value of its state or row has fewer). fp32 io: fp32
   throughout, in 16-token chunks. Deterministic. Tokens behind the last sequence are left as they
   were. `workspace`: gdn_bwd_workspace_bytes(args) bytes, 256-byte aligned. */
size_t gdn_bwd_workspace_bytes(const gdn_args *args);

kda_status gdn_bwd(const gdn_args *args, const void *d_o, const float *dht, void *workspace,
                   size_t ws_bytes, void *dq, void *dk, void *dv, void *dg, void *dbeta,
                   float *dh0, float *dA_log, float *ddt_bias, void *stream);

/* gdn_bwd with q, k and v kept as 8-bit checkpoints (act8.h): args->q, k, v are their int8 rows, q_scale,
   k_scale [B, T, H] and v_scale [B, T, HV] fp32 (4-byte aligned) the rows' scales. They are unpacked to
   the io type into the workspace; the gradients are those at these values. q, k and v together have less
   than 2^33 values. */
size_t gdn_bwd_packed_workspace_bytes(const gdn_args *args);

kda_status gdn_bwd_packed(const gdn_args *args, const float *q_scale, const float *k_scale,
                          const float *v_scale, const void *d_o, const float *dht, void *workspace,
                          size_t ws_bytes, void *dq, void *dk, void *dv, void *dg, void *dbeta,
                          float *dh0, float *dA_log, float *ddt_bias, void *stream);

/* One serving step: B rows of T new tokens each, row b on the state in slot state_indices[b]
   of `state` [slots, HV, K, V] fp32, updated in place. state_indices: device int32 [B], or
   NULL for slot b (slots >= B then). A row whose index is negative or >= slots is padding: its
   o is zero and no state is touched. Two rows must not name the same slot (their updates race).
   args: B == N, no cu_seqlens; initial_state and final_state are not read. */
kda_status gdn_step(const gdn_args *args, float *state, const int32_t *state_indices,
                    int32_t slots, void *stream);

/* Rows cu_seqlens[N] .. T - 1 of n (at most 8) tensors of T rows set to zero: those behind the last packed
   sequence, which the calls above and kda_fwd's and kda_bwd's leave as they were. x[i] device, 8-byte
   aligned, contiguous; row_bytes[i] even; both arrays on the host, read before the call returns. */
kda_status gdn_zero_tail(const int64_t *cu_seqlens, int32_t N, int64_t T, int32_t n, void *const *x,
                         const int64_t *row_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
