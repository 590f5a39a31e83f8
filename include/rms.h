/* rms.h -- C ABI of the root-mean-square norm with the residual's addition, forward (with
 * outputs of 16, 32 or 8 bits) and backward; part of libgdn.  It is the norm before and after
 * the layers of a model with gated-delta-rule layers.
 *
 * Forward, per row:
 *     h = x + residual                      (h = x without a residual)
 *     rstd = 1 / sqrt(sum_i h_i^2 / D + eps)
 *     y_i = h_i w_i rstd                    (w = 1 without a weight)
 * with y_dtype RMS_E4M3, y holds 8-bit floating point codes (e4m3: 4 exponent and 3 mantissa bits,
 * largest value 448) and scales the fp32 numbers that they are multiples of: for a row (group = 0) or for `group`
 * consecutive columns of a row,
 *     scale = max(max_i |y_i| / 448, 2^-126),   code_i = e4m3(y_i (1 / scale))
 * Backward, from the h and rstd of the forward, with n = h rstd and c = sum_i dy_i w_i n_i / D:
 *     dx_i = rstd (dy_i w_i - n_i c) + dh_i  (the gradient of x and of the residual alike; dh:
 *                                            the gradient that reaches h past the norm, may be NULL)
 *     dweight_i = sum over rows of dy_i n_i
 * Arithmetic: fp32 sums, statistics and products whatever the types; every output is rounded
 * once to its type (h included: y and rstd come from the unrounded sum).  Sums run in an order fixed by
 * rows, D and the types: results do not change from run to run, nor with alignment or strides.
 *
 * Layouts (device memory): rows of D contiguous elements.  x, residual (forward) and h, dy
 * (backward) rows are x_s, res_s elements apart; h, y, dx, dh are dense; x, residual, h, dy, dh,
 * dx have x_dtype; weight [D] has w_dtype; rstd fp32 [rows]; scales fp32 [rows] or
 * [rows][D / group]; dweight fp32 [D].  Forward: h may be the very buffer of x or of residual
 * (then that row stride must be D): the sum replaces it.
 *
 * Ownership, streams and errors are gdn.h's: work is only enqueued, nothing is allocated or kept.
 *   GDN_ERR_INVALID_ARG  NULL pointer, a negative size, D < 1, a row stride below D, unknown type, a
 *                        pointer not aligned to its element, RMS_E4M3 without scales, group not dividing D
 *   GDN_ERR_UNSUPPORTED  group not 0, 16, 32, 64 or 128; sizes beyond the kernels' index range
 *   GDN_ERR_ALIAS        an output overlaps an input (but for h, as above) or another output
 *   GDN_ERR_WORKSPACE    workspace smaller than rms_backward_workspace_bytes()
 *   GDN_ERR_CUDA         a launch failed
 */
#ifndef RMS_H
#define RMS_H

#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* y_dtype beside gdn_dtype_t's: 8-bit codes with scales. */
#define RMS_E4M3 3

typedef struct {
    int64_t rows, D;
    int64_t x_s, res_s;   /* element strides of x's and residual's rows (backward: h's and dy's) */
    int32_t x_dtype;      /* gdn_dtype_t of x, residual, h, dy, dh, dx */
    int32_t w_dtype;      /* gdn_dtype_t of weight */
    int32_t y_dtype;      /* gdn_dtype_t of y, or RMS_E4M3 */
    int32_t group;        /* RMS_E4M3: columns a scale covers; 0: the whole row */
    float eps;
    int32_t reserved0;    /* 0 */
} rms_params_t;

/* Bytes of device workspace rms_backward needs (0 when the sizes are unsupported). */
size_t rms_backward_workspace_bytes(const rms_params_t* p);

/* residual, weight, h (without it the sum is not kept), rstd may be NULL; scales only with RMS_E4M3. */
int rms_forward(const rms_params_t* p, const void* x, const void* residual, const void* weight, void* h, void* y,
                float* scales, float* rstd, void* stream);

/* weight, dh and dweight may be NULL; the workspace only serves dweight. */
int rms_backward(const rms_params_t* p, const void* h, const void* weight, const float* rstd, const void* dy,
                 const void* dh, void* dx, float* dweight, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RMS_H */
