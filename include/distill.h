/* distill.h -- C ABI of distillation from a teacher's top logits: the loss of a row of logits and its gradient; part of
 * libgdn.  Models of linear-attention and gated-delta-rule layers are taught by larger ones this way.
 *
 * Per row n, with the teacher's listed entries j < K (token indices[n][j], logit teacher[n][j]):
 *     p_j = exp(teacher_j / tau) / sum_i exp(teacher_i / tau)      over the row's entries
 *     q_w = exp(x_w / tau) / sum_w' exp(x_w' / tau)                over all V tokens of the row x = logits[n]
 *     lse[n]  = log sum_w exp(x_w / tau)
 *     loss[n] = sum_j p_j (log p_j - log q_{indices_j})
 *     dlogits[n][w] = dloss[n] / tau (q_w - sum of p_j over the entries j with indices_j = w)
 * dloss is what the loss of each row counts for (its gradient); a usual factor tau^2 belongs there.
 *   - An index outside [0, V), or a teacher's logit of -inf, is no entry: lists may be shorter than K.  A row without
 *     entries has loss and lse 0 and dlogits of zeros, whatever its logits hold.
 *   - A token listed twice counts twice.
 *   - A student's logit of -inf has q = 0: a listed one makes the loss +inf, its gradient stays finite.
 *   - NaN or +inf among a row's logits makes its loss and gradients NaN, as the formulas do; so does one among the
 *     teacher's.
 *
 * distill_forward gives loss and lse, and with dloss and dlogits the gradient in the same call: rows of up to 512 KB are
 * then read once.  distill_backward gives the gradient from the lse of an earlier forward call: of a row whose lse is beyond 32 in size, where one fp32
 * number would leave q off by 2^-24 of it, it sums the row again instead.
 *
 * Layouts (device memory): logits [N][V] in dtype, rows row_stride elements apart; dlogits in dtype, rows d_stride
 * apart, and it may be the very buffer of logits (then d_stride = row_stride): the gradient replaces them.  indices int32 [N][K],
 * teacher [N][K] in teacher_dtype, both dense; loss, lse, dloss fp32 [N].
 * Arithmetic: fp32 from the stored numbers; exponentials of the student's logits are taken of their distances to the row's largest, however far that lies from zero, and use
 * the hardware's 2^x (2^-22 relative); dlogits are rounded once.  An lse beyond fp32's range is infinite.  Sums run in an order fixed by the sizes and each row's place within 16 bytes: the same results run to run.
 *
 * Ownership, streams and errors are gdn.h's: work is only enqueued, nothing is allocated or kept.
 *   GDN_ERR_INVALID_ARG  NULL pointer, negative N or K, V < 1, a row stride below V, unknown dtype, a temperature that is not
 *                        finite or below 2^-126 (the smallest normal number), a pointer not aligned to its element, one of dloss and dlogits without the other
 *   GDN_ERR_UNSUPPORTED  K above 1024, V above 2^30, N above 2^27
 *   GDN_ERR_ALIAS        an output overlaps an input (but for dlogits, as above) or another output
 *   GDN_ERR_CUDA         a launch failed
 */
#ifndef DISTILL_H
#define DISTILL_H

#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t N, V, K;
    int64_t row_stride;     /* elements between two rows of logits */
    int64_t d_stride;       /* the same of dlogits */
    int32_t dtype;          /* gdn_dtype_t of logits and dlogits */
    int32_t teacher_dtype;  /* gdn_dtype_t of teacher */
    float temperature;      /* tau */
    int32_t reserved0;      /* 0 */
} distill_params_t;

/* dloss and dlogits may be NULL together. */
int distill_forward(const distill_params_t* p, const void* logits, const int32_t* indices, const void* teacher,
                    float* loss, float* lse, const float* dloss, void* dlogits, void* stream);

int distill_backward(const distill_params_t* p, const void* logits, const int32_t* indices, const void* teacher,
                     const float* lse, const float* dloss, void* dlogits, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DISTILL_H */
