/* beam.h -- C ABI of a beam search's selection over beams and vocabulary; part of libgdn.  With
 * gdn_decode.h it is the other half of a decoding step: the slots of the chosen parents are what
 * the next gdn_decode reads (slot_in), or what gdn_states_move copies.
 *
 * Per sequence n with K beams over V tokens, beam k's cumulative log-probability scores[n][k]:
 *     c(k, w) = scores[n][k] + (logit[n][k][w] - max) - log sum_w' exp(logit[n][k][w'] - max)
 * and the n_out best of the K V candidates, by c from high to low, equal ones by the lowest k V + w:
 *     scores_out, parent (k) and token (w); src_slots = slots[n][parent] where slots is given.
 * A finished beam (done[n][k] != 0) has one candidate: pad_token, with its score as it is.
 *   - a logit or a score that is NaN counts as -inf; a beam whose score is -inf (the unused ones
 *     of a first step) is not read, all its candidates are at -inf;
 *   - a logit of -inf (a masked token), or a row of nothing else, has candidates at -inf; they
 *     fill up, lowest index first, what too few others leave;
 *   - logits of +inf share the probability, the others have none.
 * Tokens are best masked with -inf: finite masks leave candidates like any others, and where n_out reaches into
 * thousands of equal ones, choosing among them takes milliseconds.
 * Equality is that of the fp32 c.
 *
 * Layouts (device memory): logits [N K][V] in dtype, rows row_stride elements apart, V
 * contiguous; scores fp32 [N][K]; done uint8 [N][K]; slots int32 [N][K]; outputs [N][n_out],
 * fp32 (scores_out) and int32.
 * Arithmetic: fp32 from the stored logits; sums in an order fixed by the sizes and each row's place
 * within 16 bytes, the same results run to run.
 *
 * Ownership, streams and errors are gdn.h's: work is only enqueued, nothing is allocated or
 * kept; the workspace is scratch that no call needs zeroed.
 *   GDN_ERR_INVALID_ARG  NULL pointer, negative N, K or V < 1, row_stride < V, unknown dtype, n_out
 *                        < 1 or above K V, pad_token outside [0, V) with done, a pointer not
 *                        aligned to its element (the workspace to 16 bytes), src_slots without slots
 *   GDN_ERR_UNSUPPORTED  n_out above 64, K above 64, K V or 64 N K above 2^31 - 1, more than 2^31 - 1
 *                        segments (of 32 KB of a row, or fewer where rows are few) in all
 *   GDN_ERR_ALIAS        an output or the workspace overlaps an input or another output
 *   GDN_ERR_WORKSPACE    workspace smaller than beam_workspace_bytes()
 *   GDN_ERR_CUDA         a launch failed
 */
#ifndef BEAM_H
#define BEAM_H

#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t N, K, V;
    int64_t row_stride;  /* elements between the logits of two beams */
    int32_t dtype;       /* gdn_dtype_t of the logits */
    int32_t n_out;
    int32_t pad_token;   /* what a finished beam goes on with */
    int32_t reserved0;   /* 0 */
} beam_params_t;

/* Bytes of device workspace beam_select needs (0 when the sizes are unsupported). */
size_t beam_workspace_bytes(const beam_params_t* p);

/* done, slots and src_slots may be NULL. */
int beam_select(const beam_params_t* p, const void* logits, const float* scores, const uint8_t* done,
                const int32_t* slots, float* scores_out, int32_t* parent, int32_t* token, int32_t* src_slots,
                void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BEAM_H */
