/*
 * prism_linattn.h — the linear attention layer's operators on GB300 (sm_103a): the norm
 * of query and key heads with the position rotation, and causal linear attention with
 * one decay per head (prompts, their gradients, single tokens).
 *
 * Linear attention keeps, like the mixer of prism.h, one state S [d_v, d_k] a head:
 *   S_t = exp(log_decay_h) S_{t-1} + v_t k_t^T,    o_t = scale S_t q_t.
 * It is the mixer's recurrence without the delta-rule term and the refinement, with a
 * decay fixed for each head.
 *
 * Conventions are those of prism.h (device pointers, caller-owned memory, nothing
 * allocated or kept, asynchronous on `stream`, error codes PRISM_*), except that token
 * inputs may be strided: heads of one token are contiguous ([H, d]), and `stride` gives
 * the elements from one sequence to the next (stride[0]) and from one token to the next
 * (stride[1]), so that q, k and v may lie in one fused projection.  stride[1] = 0 stands for
 * a contiguous [B,T,H,d] tensor.  Strides are multiples of 16 bytes; stride[0] is greater than 0 (a
 * sequence expanded over a batch is refused) and stride[1] is at least H*d.  Outputs are
 * contiguous and may not overlap inputs (a state in the place of one that the call still reads is
 * refused).  Pointers are 16-byte aligned; those of log_decay, positions, seq_lens and slots
 * 4-byte aligned.
 *
 *   seq_lens [B] int32 or NULL: tokens t >= seq_lens[b] are padding, as in prism.h: their
 *   outputs and gradients are 0 and their values, NaN included, reach nothing.  Lengths
 *   are clamped to 0..T.
 */
#ifndef PRISM_LINATTN_H
#define PRISM_LINATTN_H

#include "prism.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Norm of query and key heads, with the position rotation ---- */

#define PRISM_ROPE_INTERLEAVED 1u /* pairs (2i, 2i+1); without it (i, i + rotary_dim/2) */

typedef struct {
    int B, T;
    int Hq, Hk;            /* query heads and key heads */
    int d;                 /* head dim: 16, 32, 64 or 128 */
    int rotary_dim;        /* r: the first r dims of a head turn; a multiple of 8, 0 <= r <= d */
    int table_rows;        /* positions 0..table_rows-1 have an angle */
    prism_dtype dtype;     /* type of q, k and of the outputs */
    unsigned flags;        /* PRISM_ROPE_* */
    float eps;             /* >= 0 */
    float q_scale, k_scale;
    long long q_stride[2], k_stride[2];     /* of q and k */
    long long dq_stride[2], dk_stride[2];   /* of the gradients that come in (backward) */
} prism_rope_dims;

/* For each head vector x of q (and of k, with k_weight and k_scale):
 *   n = x / sqrt(mean(x^2) + eps),   y = rotate(q_scale * q_weight * n)
 * where rotate turns pair i by the angle whose cosine and sine are table[p][i] and
 * table[p][r/2 + i] at the token's position p, and leaves dims r..d-1.  The mixer's unit
 * norm is q_scale = d^-1/2 with eps/d for eps and no weight.
 *   q_weight, k_weight  [d] fp32, or NULL (ones)
 *   table      [table_rows, r] fp32 (may be NULL when r = 0)
 *   positions  [B,T] int32, or NULL: position t (then table_rows >= T when r > 0).  A
 *              token whose position is outside 0..table_rows-1 is padding (when r > 0).
 *   q_out, k_out  [B,T,Hq,d], [B,T,Hk,d]
 * Arithmetic is fp32, rounded once. */
PRISM_API int prism_qk_norm_rope(const prism_rope_dims* dims, const void* q, const void* k,
                                 const float* q_weight, const float* k_weight, const float* table,
                                 const int32_t* positions, const int32_t* seq_lens,
                                 void* q_out, void* k_out, void* stream);

/* Gradients through prism_qk_norm_rope: dq_out, dk_out are the gradients of its outputs
 * (in dtype, strided as dims say), dq, dk those of q and k (in dtype, contiguous);
 * dq_weight, dk_weight [d] fp32 are overwritten (either may be NULL: not wanted).  Sums
 * over tokens and heads run in a fixed order (no atomics).  The workspace
 * (prism_qk_norm_rope_workspace_bytes) is scratch, 256-byte aligned. */
PRISM_API size_t prism_qk_norm_rope_workspace_bytes(const prism_rope_dims* dims);
PRISM_API int prism_qk_norm_rope_backward(const prism_rope_dims* dims, const void* q, const void* k,
                                          const float* q_weight, const float* k_weight,
                                          const float* table, const int32_t* positions,
                                          const int32_t* seq_lens, const void* dq_out,
                                          const void* dk_out, void* dq, void* dk,
                                          float* dq_weight, float* dk_weight, void* workspace,
                                          size_t workspace_bytes, void* stream);

/* ---- Linear attention with a decay per head ---- */

typedef struct {
    int B, T, H;
    int d;                 /* d_k = d_v: 16, 32, 64 or 128 */
    prism_dtype dtype;     /* type of q, k, v, out and their gradients */
    unsigned flags;        /* 0 or PRISM_FLAG_CHECK_WAIT_TIMEOUT */
    float scale;
    long long q_stride[2], k_stride[2], v_stride[2];
    long long do_stride[2];                 /* of d_out (backward) */
} prism_linattn_dims;

/* Prompts, in chunks: out [B,T,H,d] in dtype; final_state [B,H,d_v,d_k] fp32 (NULL: not
 * written) after each sequence's last token; initial_state (NULL: zero) before its first.
 *   log_decay  [H] fp32, <= 0 (-inf: no memory at all)
 * A non-finite value reaches what comes after it (outputs, in the gradients what comes after in their
 * own direction, and states) as in the recurrence, and nothing before it.  What has decayed below
 * 2^-126, fp32's smallest normal number, may count as nothing, a non-finite value's share
 * as well.  Sums and states are fp32.  In PRISM_BF16 the products run on the tensor
 * cores: scores and the state that a chunk reads are rounded to bf16 once; the state's own
 * update keeps 16 bits of the decayed key (two bf16 terms), and 24 (three) in the tokens that
 * final_state, or the backward pass's d_initial_state, remembers by more than a quarter. */
PRISM_API size_t prism_linattn_workspace_bytes(const prism_linattn_dims* dims);
PRISM_API int prism_linattn_forward(const prism_linattn_dims* dims, const void* q, const void* k,
                                    const void* v, const float* log_decay,
                                    const float* initial_state, void* out, float* final_state,
                                    const int32_t* seq_lens, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* Gradients through prism_linattn_forward, given d_out [B,T,H,d] in dtype and d_final_state
 * [B,H,d_v,d_k] fp32 (NULL: zero): dq, dk, dv in dtype; d_initial_state fp32 (NULL: not
 * wanted).  log_decay is a constant of the layer and gets no gradient.  Deterministic. */
PRISM_API size_t prism_linattn_backward_workspace_bytes(const prism_linattn_dims* dims);
PRISM_API int prism_linattn_backward(const prism_linattn_dims* dims, const void* q, const void* k,
                                     const void* v, const float* log_decay,
                                     const float* initial_state, const void* d_out,
                                     const float* d_final_state, void* dq, void* dk, void* dv,
                                     float* d_initial_state, const int32_t* seq_lens,
                                     void* workspace, size_t workspace_bytes, void* stream);

/* One token of every sequence (dims->T = 1): q, k, v [B,H,d], out [B,H,d] in dtype.
 *   state  [n_states,H,d_v,d_k] fp32, updated in place
 *   slots  [B] int32, or NULL (state b belongs to sequence b, n_states >= B).  A sequence
 *          whose slot is outside 0..n_states-1 is not there: its out is 0 and no state
 *          moves.  Two sequences may not share a slot. */
PRISM_API int prism_linattn_decode_step(const prism_linattn_dims* dims, const void* q, const void* k,
                                        const void* v, const float* log_decay, float* state,
                                        int n_states, const int32_t* slots, void* out,
                                        void* stream);

/* Failure detection: the waits of the tensor-core kernels on copies and products are
 * bounded; one that gives up sets the library's word for the current device, which stays
 * set until it is cleared.  Synchronises the device and returns the word in *word (0: no
 * wait gave up), clearing it when `clear` is nonzero.  PRISM_ERR_INVALID_ARG for a NULL
 * word, PRISM_ERR_CUDA when the synchronisation or the copy fails.
 *
 * A wait's limit is about a second.  PRISM_FLAG_CHECK_WAIT_TIMEOUT in dims->flags is a diagnostic
 * of this path: in prism_linattn_forward and _backward on the PRISM_BF16 path (it is ignored on
 * PRISM_F32 and refused by prism_linattn_decode_step) the copies of every CTA with tokens first
 * wait, for a millisecond, for what never comes, and give up.  The roles that wait for them
 * follow after their second, the call returns, the word is set and its outputs are undefined. */
PRISM_API int prism_linattn_status(int* word, int clear);

#ifdef __cplusplus
}
#endif
#endif /* PRISM_LINATTN_H */
