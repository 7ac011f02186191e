/*
 * prism_gated.h — the gated recurrent layer's operators on GB300 (sm_103a): layer norm over a
 * token's whole width, and the gated linear recurrence with a gate for every channel and token
 * (prompts, their gradients, single tokens).
 *
 * The recurrence keeps one number h a channel:
 *   h_t = a_t h_{t-1} + w_t x_t,   out_t = h_t,   a_t = sigmoid(forget_t),
 *   w_t = sigmoid(input_gate_t), or 1 - a_t where there is no input gate.
 * It is the mixer's recurrence (prism.h) with a state as wide as the token instead of d_v x d_k a
 * head, and a forget gate for every channel of it.
 *
 * Conventions are those of prism.h (device pointers, caller-owned memory, nothing allocated or
 * kept, asynchronous on `stream`, error codes PRISM_*), except that token inputs may be strided:
 * the D channels of one token are contiguous, and `stride` gives the elements from one sequence to
 * the next (stride[0]) and from one token to the next (stride[1]), so that x and the gates may lie
 * in one fused projection.  stride[1] = 0 stands for a contiguous [B,T,D] tensor.  Strides are
 * multiples of 16 bytes; stride[0] is greater than 0 (a sequence expanded over a batch is
 * refused) and stride[1] is at least D.  Outputs are contiguous and may not overlap inputs or one
 * another, but for a state that is written over the one that came in (below).  Pointers are
 * 16-byte aligned; those of seq_lens and slots 4-byte aligned, workspaces 256-byte.  A workspace
 * is scratch for one call: two calls that may run at the same time take one each.
 *
 *   D   channels of a token: a multiple of 8 up to 2^30 (layer norm: up to 16384)
 *   T   up to 2^30 tokens, B * T below 2^31
 *   seq_lens [B] int32 or NULL: tokens t >= seq_lens[b] are padding, as in prism.h: their
 *   outputs and gradients are 0 and their values, NaN included, reach nothing.  Lengths
 *   are clamped to 0..T.
 */
#ifndef PRISM_GATED_H
#define PRISM_GATED_H

#include "prism.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Layer norm ---- */

typedef struct {
    int B, T, D;
    prism_dtype dtype;     /* type of x, out and the gradients of tokens */
    unsigned flags;        /* 0 */
    float eps;             /* >= 0 */
    long long x_stride[2];
    long long do_stride[2];    /* of d_out (backward) */
} prism_layer_norm_dims;

/* For each token x [D]:  out = (x - mean(x)) / sqrt(var(x) + eps) * weight + bias,
 * var(x) = mean((x - mean(x))^2).
 *   weight, bias [D] fp32, or NULL (ones, zeros)
 *   out          [B,T,D] in dtype
 * The mean comes before the squares (no difference of large sums); arithmetic is fp32, rounded once. */
PRISM_API int prism_layer_norm(const prism_layer_norm_dims* dims, const void* x, const float* weight,
                               const float* bias, const int32_t* seq_lens, void* out, void* stream);

/* Gradients through prism_layer_norm, given d_out [B,T,D] in dtype: dx in dtype, d_weight and
 * d_bias [D] fp32 overwritten (either may be NULL: not wanted).  Sums over tokens run in a fixed
 * order (no atomics).  The workspace (prism_layer_norm_workspace_bytes) is needed for d_weight and
 * d_bias and may be NULL where neither is wanted. */
PRISM_API size_t prism_layer_norm_workspace_bytes(const prism_layer_norm_dims* dims);
PRISM_API int prism_layer_norm_backward(const prism_layer_norm_dims* dims, const void* x, const float* weight,
                                        const int32_t* seq_lens, const void* d_out, void* dx, float* d_weight,
                                        float* d_bias, void* workspace, size_t workspace_bytes, void* stream);

/* ---- Gated linear recurrence ---- */

#define PRISM_GATED_CHUNK 64   /* tokens from one row of `states` to the next */

typedef struct {
    int B, T, D;
    prism_dtype dtype;     /* type of x, the gates, out and their gradients */
    unsigned flags;        /* 0 or PRISM_FLAG_CHECK_WAIT_TIMEOUT */
    long long x_stride[2], f_stride[2], i_stride[2];   /* of x, forget and input_gate */
    long long do_stride[2];                            /* of d_out (backward) */
} prism_gated_dims;

/* Prompts: out [B,T,D] in dtype; final_state [B,D] fp32 (NULL: not written) after each sequence's
 * last token; initial_state (NULL: zero) before its first.  final_state may be initial_state.
 *   input_gate  [B,T,D], or NULL: w_t = 1 - a_t
 *   states      [B, ceil(T/64), D] fp32, or NULL: the state before the tokens 0, 64, 128, ... of each
 *               sequence, which prism_gated_scan_backward reads.  Rows that start at or behind a
 *               sequence's end are left as they are.
 * Gates and states are fp32; out is rounded once.  A gate below 2^-126 counts as 0, and so may a
 * product of gates below it (an infinite state may become NaN there).  Tiles of a
 * sequence wait for the state of the tiles before them; the result does not depend on their
 * timing (two calls agree bit for bit).  The workspace has prism_gated_scan_workspace_bytes (0 where
 * no tile looks back: it may then be NULL). */
PRISM_API size_t prism_gated_scan_workspace_bytes(const prism_gated_dims* dims);
PRISM_API int prism_gated_scan_forward(const prism_gated_dims* dims, const void* x, const void* forget,
                                       const void* input_gate, const float* initial_state, void* out,
                                       float* final_state, float* states, const int32_t* seq_lens,
                                       void* workspace, size_t workspace_bytes, void* stream);

/* Gradients through prism_gated_scan_forward, given its inputs, the `states` that it wrote, d_out
 * [B,T,D] in dtype and d_final_state [B,D] fp32 (NULL: zero): dx, d_forget and d_input_gate (NULL
 * without an input gate, and only then) in dtype; d_initial_state [B,D] fp32 (NULL: not wanted), which
 * may be d_final_state.  Deterministic. */
PRISM_API size_t prism_gated_scan_backward_workspace_bytes(const prism_gated_dims* dims);
PRISM_API int prism_gated_scan_backward(const prism_gated_dims* dims, const void* x, const void* forget,
                                        const void* input_gate, const float* states, const void* d_out,
                                        const float* d_final_state, void* dx, void* d_forget,
                                        void* d_input_gate, float* d_initial_state, const int32_t* seq_lens,
                                        void* workspace, size_t workspace_bytes, void* stream);

/* One token of every sequence (dims->T = 1): x, forget, input_gate (or NULL), out [B,D] in dtype.
 *   state  [n_states,D] fp32, updated in place
 *   slots  [B] int32, or NULL (state b belongs to sequence b, n_states >= B).  A sequence
 *          whose slot is outside 0..n_states-1 is not there: its out is 0 and no state
 *          moves.  Two sequences may not share a slot. */
PRISM_API int prism_gated_scan_decode_step(const prism_gated_dims* dims, const void* x, const void* forget,
                                           const void* input_gate, float* state, int n_states,
                                           const int32_t* slots, void* out, void* stream);

/* Failure detection: a tile's look back for the state before it, and a kernel's waits for its own copies, are
 * bounded (about a second); one that gives up sets the library's word for the current device, which stays
 * set until it is cleared, and the call's outputs are then undefined.  (Where the tiles of a sequence are the
 * CTAs of a cluster, they meet at its barrier, which has no limit of its own: the CTAs of a cluster run at the same time, and
 * each gets there behind bounded waits alone.)  Synchronises the device and returns the word in *word (0: no
 * wait gave up), clearing it when `clear` is nonzero.  PRISM_ERR_INVALID_ARG for a NULL word,
 * PRISM_ERR_CUDA when the synchronisation or the copy fails.
 *
 * PRISM_FLAG_CHECK_WAIT_TIMEOUT in dims->flags is a diagnostic of the look back (refused by
 * prism_gated_scan_decode_step): every tile that looks back first waits, for a millisecond, for what
 * never comes, and gives up.  The word is set; the outputs are then computed as without the flag.  Where no
 * tile looks back (a call that needs no workspace, sequences of one tile) the flag does nothing. */
PRISM_API int prism_gated_status(int* word, int clear);

#ifdef __cplusplus
}
#endif
#endif /* PRISM_GATED_H */
