/* gdn_decode.h -- C ABI of the gated delta rule's serving form: the recurrence over a pool of
 * states, a few tokens a sequence, and the moves of states between the pool's slots.  Part of
 * libgdn; the rule, its sources and its key-head mapping (h mod H_k) are those of gdn.h.
 *
 * What is computed, per sequence n, value head h and token t of the sequence, with a = exp(g):
 *     S'  = a (.) M_{t-1};   delta_j = beta (v_j - sum_i S'[j][i] k_i)
 *     M_t = S' + delta k^T;  y_j = scale sum_i M_t[j][i] q_i
 * M_0 is the state in slot slot_in[n] of the pool (zero where slot_in[n] is -1), and the state
 * after the sequence's last token goes to slot slot_out[n] (nowhere where it is -1).  A sequence
 * without tokens copies its state.  Equal slots update in place; another slot_out keeps the
 * state before the step, so that drafted tokens can be taken back or the children of one beam
 * can start from one parent's slot.
 *
 * Layouts (device memory)
 *   q, k   [n_tok][H_k][S_k]  element strides q_s/k_s = {token, head}, head elements contiguous
 *   v      [n_tok][H_v][S_v]  strides v_s, head elements contiguous (row views of a packed qkv buffer are fine)
 *   g      [n_tok][H_v] (scalar gate) or [n_tok][H_v][S_k] (KDA), beta [n_tok][H_v]; contiguous, in gate_dtype
 *   y      [n_tok][H_v][S_v] contiguous, in y_dtype
 *   cu_tokens  int32 [n_seq + 1]: sequence n owns the token rows cu_tokens[n] .. cu_tokens[n+1]-1;
 *              NULL: every sequence has T tokens, n_tok = n_seq T
 *   pool   [n_slots][H_v][S_v][S_k] fp32, slots slot_stride elements apart
 *   slot_in, slot_out  int32 [n_seq]
 * Arithmetic: states, products, sums and gates are fp32 (accurate expf, no fast-math) whatever
 * the types; y is rounded once to y_dtype.  Results do not depend on the batch or the launch.
 *
 * Within one call, a slot that a sequence writes must not be read or written by another
 * sequence (several may read one slot).  Rows of q .. y that no sequence owns are left alone.
 *
 * A slot outside [-1, n_slots) or a cu_tokens that falls, or leaves [0, n_tok], is only seen on the
 * device: the kernel skips that sequence (its rows of y and its slot keep what they held) and
 * the next gdn_device_status returns GDN_ERR_INVALID_ARG.
 *
 * Ownership, streams and errors are those of gdn.h: work is only enqueued on `stream`, nothing
 * is allocated or kept, no output is written when a call returns an error.
 *   GDN_ERR_INVALID_ARG  NULL pointer, a negative size or stride, H_v % H_k != 0, n_tok != n_seq T
 *                        without cu_tokens, unknown gate or dtype, a pool that is not 16-byte aligned or
 *                        whose slot_stride is not a multiple of 4 of at least H_v S_v S_k, an input
 *                        not aligned to its element
 *   GDN_ERR_UNSUPPORTED  S_k not one of 16, 32, 64, 128, 256; S_v not a multiple of 16 up to 256;
 *                        sizes beyond the kernels' index range
 *   GDN_ERR_ALIAS        y or the pool overlaps an input or the other
 *   GDN_ERR_CUDA         a launch failed
 */
#ifndef GDN_DECODE_H_
#define GDN_DECODE_H_

#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t n_seq, T, n_tok;          /* sequences; tokens of each without cu_tokens; token rows */
    int64_t H_k, H_v, S_k, S_v;       /* as in gdn_params_t */
    int64_t n_slots, slot_stride;     /* the pool's slots, and the elements from one to the next */
    int64_t q_s[2], k_s[2], v_s[2];   /* element strides of {token, head} */
    int32_t gate;                     /* gdn_gate_t */
    int32_t in_dtype;                 /* gdn_dtype_t of q, k, v */
    int32_t gate_dtype;               /* gdn_dtype_t of g, beta */
    int32_t y_dtype;                  /* gdn_dtype_t of y */
    float scale;                      /* output scale, usually 1/sqrt(S_k) */
    int32_t reserved0;                /* 0 */
} gdn_decode_params_t;

/* GDN_OK when the sizes and types are supported, else the code gdn_decode would return. */
gdn_status_t gdn_decode_supported(const gdn_decode_params_t* p);

gdn_status_t gdn_decode(const gdn_decode_params_t* p, const void* q, const void* k, const void* v, const void* g,
                        const void* beta, const int32_t* cu_tokens, float* pool, const int32_t* slot_in,
                        const int32_t* slot_out, void* y, void* stream);

/* Moves of states between slots, in every layer's pool at once: for each move i,
 * slot dst[i] = what slot src[i] held before the call, or zeros where src[i] is -1; a move with
 * dst[i] = -1 or dst[i] = src[i] does nothing.  Copying, forking (one source, several
 * destinations), freeing to zero, compacting, and a beam search's reordering are lists of moves.
 *
 * The moves are taken `group` at a time (moves 0 .. group-1, group .. 2 group-1, ...; the last
 * group may be short).  Inside a group they are simultaneous: any of its slots may be source and
 * destination at once, as when beams change places.  Different groups must not write a slot that
 * the other reads or writes, and no two moves write one slot.
 *
 *   pool   device memory: layer l's slot s starts at pool + l layer_stride + s slot_stride (bytes)
 *          and holds state_bytes; everything 16-byte aligned (any contents: states, windows)
 *   src, dst   int32 [n_moves], device memory
 * A slot outside [-1, n_slots) skips its move and is reported by gdn_device_status, as above.
 *
 *   GDN_ERR_INVALID_ARG  NULL pointer, negative size, misalignment, strides that overlap slots, group < 1
 *   GDN_ERR_UNSUPPORTED  group above 1024
 *   GDN_ERR_ALIAS        src or dst inside the pool
 *   GDN_ERR_CUDA         a launch failed */
gdn_status_t gdn_states_move(void* pool, int64_t n_layers, int64_t layer_stride, int64_t n_slots, int64_t slot_stride,
                             int64_t state_bytes, const int32_t* src, const int32_t* dst, int64_t n_moves,
                             int64_t group, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_DECODE_H_ */
