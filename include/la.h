/* la.h -- C ABI of linear attention with a decay for each head, forward (prompts and single tokens
 * over a pool of states) and backward; part of libgdn.  It is the gated delta rule (gdn.h) without the correction:
 * layers of both kinds stand in one model, share gdn.h's key-head mapping (h mod H_k) and gdn_decode.h's pools.
 *
 * What is computed, per sequence n, value head h and token t of the sequence, with a_t = exp(g_t):
 *     M_t = a_t M_{t-1} + v_t k_t^T;   y_t = scale M_t q_t                  (M: S_v x S_k)
 * M_0 is the state in slot slot_in[n] of the pool (zero where slot_in[n] is -1), and the state after the
 * sequence's last token goes to slot slot_out[n] (nowhere where it is -1).  A sequence without tokens copies its
 * state.  Equal slots update in place.
 * Backward, from dy, the gradient dM_T that reaches the last state (may be NULL: zero), and M_0 as above:
 *     D_T = dM_T + scale dy_T q_T^T;   D_t = a_{t+1} D_{t+1} + scale dy_t q_t^T
 *     dq_t = scale M_t^T dy_t;   dk_t = D_t^T v_t;   dv_t = D_t k_t;   dg_t = a_t <D_t, M_{t-1}>;   dM_0 = a_1 D_1
 * dq and dk are sums over the value heads that share a key head.  Without tokens dM_0 = dM_T.
 *
 * Two forms compute this (la_form() says which runs):
 *   - the token form walks token by token, states in registers: every type and size;
 *   - the chunked form (bf16, S_k = S_v = 64 or 128, T of 32 or more; of many heads of 64, 48) takes 128 tokens at a time as dense products on the tensor
 *     cores, and long sequences in segments whose states are joined, so that a single prompt fills the GPU.
 *
 * Layouts (device memory)
 *   q, k   [n_tok][H_k][S_k]  element strides q_s/k_s = {token, head}, head elements contiguous
 *   v      [n_tok][H_v][S_v]  strides v_s (row views of a packed qkv buffer are fine)
 *   g      log decays [n_tok][H_v] in gate_dtype, strides g_s = {token, head}; token stride 0: one decay a head
 *   y, dy  [n_tok][H_v][S_v] contiguous; y in y_dtype, dy in in_dtype
 *   dq, dk [n_tok][H_k][S_k], dv [n_tok][H_v][S_v] contiguous, in in_dtype; dg fp32 [n_tok][H_v] contiguous, whatever g's strides
 *   dstate_T, dstate_0  fp32 [n_seq][H_v][S_v][S_k], 16-byte aligned
 *   cu_tokens  int32 [n_seq + 1]: sequence n owns the token rows cu_tokens[n] .. cu_tokens[n+1]-1, T of them at most;
 *              NULL: every sequence has T tokens, n_tok = n_seq T
 *   pool   [n_slots][H_v][S_v][S_k] fp32, slots slot_stride elements apart
 *   slot_in, slot_out  int32 [n_seq]
 * Arithmetic: states and sums are fp32 whatever the types.  The token form adds (e^g - 1) times a state to it (CUDA's expm1f; beyond half
 * a token's memory e^g times it, expf), so that a decay's rounding does not add up over the tokens that a state remembers; an infinite state may become NaN by it; the backward pass takes dq and dk in it always, by
 * segments whose first states the chunked form makes where it fits, and dv in the form that la_form() says.  The chunked form's products take bf16
 * inputs as they are and fp32 operands (states, weighted scores, decayed keys) as the sum of two bf16 numbers, 2^-16 relative,
 * with fp32 accumulation, whose sums are cut off, not rounded: a state that remembers n chunks of 128 tokens loses up to n 2^-22 of itself by it (65536 tokens 1.3e-4), where the
 * token form rounds at random; its sums of log decays are exact in 64-bit fixed point (2^-31 powers of two), each exponential of a difference the
 * hardware's 2^x (2^-22 relative).  Outputs are rounded once.
 * dg is a running sum over the tokens that follow, anchored by <M_T, dM_T>: its error is that of the sum, not of
 * the element.  Log decays below -104 (exp = 0 in fp32) count as a = 0.  The same call gives the same bits; in the chunked form
 * they depend on n_seq, T and H_v through the segments.
 *
 * An infinity or NaN in a token's inputs reaches what the formulas say, and in the chunked form also the other outputs (y and dv) of the chunk of 128
 * tokens that it lies in, y's counted from the sequence's first token, dv's from its last (a masked weight of zero is still multiplied).  dg is a running
 * sum over the tokens that follow, so what makes a token's dq or dk infinite or NaN reaches dg of every earlier token of the sequence and value head too.  Never
 * another sequence, nor, in the token form, an earlier token's y.
 * Decays that grow (g > 0) are fine as long as their products stay within fp32.
 *
 * Within one call, a slot that a sequence writes must not be read or written by another sequence (several may read
 * one slot).  Rows that no sequence owns are left alone in every output.
 *
 * A slot outside [-1, n_slots), a cu_tokens that falls, leaves [0, n_tok] or gives a sequence more than T tokens is only seen
 * on the device: that sequence is skipped (its outputs keep what they held; in the backward pass, its gradients are unspecified, and where cu_tokens
 * falls or leaves [0, n_tok], those of the whole call)
 * and the next gdn_device_status returns GDN_ERR_INVALID_ARG; GDN_ERR_TIMEOUT where one of the chunked form's bounded waits gave up.
 *
 * Ownership, streams and errors are those of gdn.h: work is only enqueued on `stream`, nothing is allocated or kept, no
 * output is written when a call returns an error; workspaces are scratch that no call needs zeroed.
 *   GDN_ERR_INVALID_ARG  NULL pointer, a negative size or stride, H_v % H_k != 0, n_tok != n_seq T
 *                        without cu_tokens, unknown dtype, a pool or workspace that is not 16-byte aligned, a
 *                        slot_stride that is not a multiple of 4 of at least H_v S_v S_k, an input not aligned to its element
 *   GDN_ERR_UNSUPPORTED  S_k not one of 16, 32, 64, 128, 256; S_v not a multiple of 16 up to 256 (backward: not one
 *                        of S_k's); sizes beyond the kernels' index range
 *   GDN_ERR_ALIAS        an output, the pool or the workspace overlaps an input or another of them (y may not be v)
 *   GDN_ERR_WORKSPACE    workspace smaller than la_workspace_bytes() / la_backward_workspace_bytes()
 *   GDN_ERR_CUDA         a launch failed
 */
#ifndef LA_H
#define LA_H

#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t n_seq, T, n_tok;                  /* sequences; tokens of the longest (of each without cu_tokens); token rows */
    int64_t H_k, H_v, S_k, S_v;               /* as in gdn_params_t */
    int64_t n_slots, slot_stride;             /* the pool's slots, and the elements from one to the next */
    int64_t q_s[2], k_s[2], v_s[2], g_s[2];   /* element strides of {token, head} */
    int32_t in_dtype;                         /* gdn_dtype_t of q, k, v, dy, dq, dk, dv */
    int32_t gate_dtype;                       /* gdn_dtype_t of g */
    int32_t y_dtype;                          /* gdn_dtype_t of y */
    float scale;                              /* output scale, usually 1/sqrt(S_k) */
} la_params_t;

/* 0: token form, 1: chunked form, -1: unsupported sizes or types. */
int la_form(const la_params_t* p);

/* Bytes of device workspace (may be 0; also 0 when the sizes are unsupported). */
size_t la_workspace_bytes(const la_params_t* p);
size_t la_backward_workspace_bytes(const la_params_t* p);

int la_forward(const la_params_t* p, const void* q, const void* k, const void* v, const void* g,
               const int32_t* cu_tokens, float* pool, const int32_t* slot_in, const int32_t* slot_out, void* y,
               void* workspace, size_t workspace_bytes, void* stream);

/* Diagnostic: la_forward (chunked form) with one of its kernels' hand-overs withheld, so that bounded waits run out, the kernels wait for their copies and products in
 * flight and return, and the next gdn_device_status is GDN_ERR_TIMEOUT.  y is unspecified, the pool keeps what it held
 * (but for sequences without tokens, which wait for nothing). */
int la_selftest_wait_timeout(const la_params_t* p, const void* q, const void* k, const void* v, const void* g,
                             const int32_t* cu_tokens, float* pool, const int32_t* slot_in, const int32_t* slot_out, void* y,
                             void* workspace, size_t workspace_bytes, void* stream);

/* slot_in and the pool as the forward found them (M_0 unchanged).  dstate_T and dstate_0 may be NULL. */
int la_backward(const la_params_t* p, const void* q, const void* k, const void* v, const void* g,
                const int32_t* cu_tokens, const float* pool, const int32_t* slot_in, const void* dy,
                const float* dstate_T, void* dq, void* dk, void* dv, float* dg, float* dstate_0,
                void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LA_H */
