/*
 * glr.h -- C ABI of libkda_fwd: the gated linear recurrence with one state a channel, on one AMD
 * Instinct MI355X (gfx950).
 *
 * The operation: for every sequence s and channel d, with a state h that starts at
 * initial_state[s, d] (or zero), each token t does
 *
 *     h <- exp(g[t, d]) h + beta[t, d] x[t, d];   y[t, d] = h
 *
 * and final_state[s, d] is h after the last token (initial_state for a sequence of no tokens).
 *
 * Conventions are kda_fwd.h's: device pointers, caller-owned; nothing is allocated, nothing
 * synchronises, results are deterministic (the numbers that a long sequence's tiles take are the only
 * atomics), errors only through the return value; concurrent calls use distinct workspaces and outputs.
 * A tensor's channels are contiguous. x, g and beta may be columns of wider rows (x_stride and so on:
 * elements from one token to the next) and some tokens of a longer batch (x_batch and so on: from one
 * sequence's first token to the next's); everything else is contiguous. io tensors are aligned to their
 * elements, fp32 tensors to 4 bytes, cu_seqlens to 8.
 *
 * Numbers. A NaN or an infinity reaches its own channel of its own sequence, from its token on (in the
 * backward: up to it). Behind its token an infinity is an infinity or a NaN: decays are applied as e^g - 1 and
 * as products, so that e^g times infinity may come out as infinity minus infinity or zero times it.
 * Log decays above zero are taken too, with e^g rounded to 24 bits, while their sums over up to 1024
 * neighbouring tokens stay below 88; beyond, where e^88 overflows, states may become NaN even where they are
 * zero. Final states, dh0, dA_log and ddt_bias are fp32 for either io and err by about 1e-7 of themselves; for
 * bf16 io a channel that decays by about 2^-8 a token for long may err by up to 2^-17. The last bits of a
 * channel may depend on the decays of the channels beside it (which form of a decay a wave takes).
 */
#ifndef GLR_H
#define GLR_H

#include <stddef.h>
#include <stdint.h>

#include "kda_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    /* A dense batch has N == B sequences of T tokens; with cu_seqlens B == 1 and sequence s spans
       [cu_seqlens[s], cu_seqlens[s + 1]), as in kda_fwd_args.                                       */
    int32_t B, T, N;
    int32_t D;                /* channels                                                            */
    int32_t io;               /* kda_dtype of x, g, beta, y (and of the gradients)                   */
    const void *x;            /* [B, T, D]                                                           */
    const void *g;            /* [B, T, D]  log decay; any g <= 0 is exact to rounding, -inf (which
                                 clears the state) included                                          */
    const void *beta;         /* [B, T, D], or NULL for ones                                         */
    int64_t x_stride, g_stride, beta_stride;
    const int64_t *cu_seqlens;/* device [N + 1] or NULL                                              */
    const float *initial_state; /* [N, D] fp32, or NULL for zeros                                    */
    void *y;                  /* [B, T, D]                                                           */
    float *final_state;       /* [N, D] fp32, or NULL to skip; may be the buffer of initial_state    */
    /* Pre-stage (all zero: inputs used as given):
         beta_sigmoid  beta <- 1 / (1 + exp(-beta))
         gate          with u = g[t, d] + dt_bias[d]: KDA_GATE_SOFTPLUS
                       g <- -exp(A_log[d]) log(1 + exp(u)); KDA_GATE_BOUNDED
                       g <- lower_bound / (1 + exp(-exp(A_log[d]) u))                                */
    int32_t beta_sigmoid, gate;
    float gate_lower_bound;   /* KDA_GATE_BOUNDED: finite and < 0                                    */
    const float *A_log;       /* [D] fp32; required for a gate                                       */
    const float *dt_bias;     /* [D] fp32, or NULL for zeros                                         */
    /* Dense batches: elements from one sequence's first token to the next's, at least (T - 1) token strides
       and D; 0: T token strides. Not read for B == 1.                                               */
    int64_t x_batch, g_batch, beta_batch;
} glr_args;

/* Bytes of device workspace glr_fwd / glr_bwd need (only shapes, io, gate, whether beta and cu_seqlens
   are there, and the current device's compute-unit count are read): may be 0, and is 0 where these are
   invalid or unsupported by themselves. Its contents need not be kept between calls. */
size_t glr_fwd_workspace_bytes(const glr_args *args);
size_t glr_bwd_workspace_bytes(const glr_args *args);

/* Enqueue the forward on `stream`: strips of channels that take a sequence in one workgroup each, or for
   long sequences tiles of 64 or 128 tokens that hand states to each other within the launch (they wait for tiles
   that have begun only). States and sums are fp32; results do not depend on the order in which tiles run.
   A wait that is not met within about a tenth of a second, which only a workspace in use by another call
   at once or decreasing offsets can bring about, ends with NaN in the states behind it (the call has
   returned KDA_OK by then). Outputs overlap no inputs but final_state its initial_state.
   Tokens behind the last sequence are left as they were. D and the strides from token to token are at most 2^18.
   A launch has fewer than 2^23 workgroups, or the call is KDA_ERR_UNSUPPORTED: about N ceil(D / 64) for strips where
   sequences are many, at most (B T / 64 + N) ceil(D / 64) for tiles. */
kda_status glr_fwd(const glr_args *args, void *workspace, size_t ws_bytes, void *stream);

/* Gradients of glr_fwd's inputs from the gradients of a loss with respect to y (d_y, like y) and to
   final_state (dht, fp32 [N, D], or NULL for zero). args as for glr_fwd, with y its output as it was
   written: h[t - 1] is read from it (final_state is not read, and x only with beta). Written:
     dx, dg            [B, T, D] io dtype, of the raw inputs
     dbeta             likewise; with beta only
     dh0               [N, D] fp32, or NULL to skip; may be the buffer of dht
     dA_log, ddt_bias  [D] fp32: with a gate, dA_log required, ddt_bias or NULL; ignored without
   Deterministic. Tokens behind the last sequence are left as they were. Outputs overlap no inputs but dh0 its dht. */
kda_status glr_bwd(const glr_args *args, const void *d_y, const float *dht, void *workspace, size_t ws_bytes,
                   void *dx, void *dg, void *dbeta, float *dh0, float *dA_log, float *ddt_bias, void *stream);

/* One serving step: B rows of T new tokens each, row b on the state in slot state_indices[b] of
   `state` [slots, D] fp32, updated in place. state_indices: device int32 [B], or NULL for slot b
   (slots >= B then). A row whose index is negative or >= slots is padding: its y is zero and no state
   is touched. Two rows must not name the same slot (their updates race). args: B == N, no cu_seqlens;
   initial_state and final_state are not read. */
kda_status glr_step(const glr_args *args, float *state, const int32_t *state_indices, int32_t slots,
                    void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GLR_H */
