// distill_internal.h -- what distillation's two kernels share (include/distill.h).
#pragma once

#include <cuda_runtime.h>

#include "../../include/distill.h"

namespace gdn {

enum { kLoss = 0, kBoth = 1, kGradient = 2 };

struct DistillArgs {
    const void* logits;
    const int* indices;
    const void* teacher;
    float *loss, *lse;
    const float *lse_in, *dloss;
    void* dlogits;
    long long row_stride, d_stride;
    int V, K, seg, chunks, ctas, teacher_dtype;
    float inv_tau, L;
};

// An lse beyond this (its size) is not what the gradient alone goes by: one fp32 number leaves q off by 2^-24 of it.  The row's largest logit and sum are taken again, from the
// same reading.
constexpr float kMostLse = 32.f;

#if defined(__CUDACC__)
// What is taken off a row's logits before they are multiplied by L: the largest, m, since 2^(x L - m L) with m L rounded would be off by half an ulp of m L powers of
// two; nothing of a row of -inf (and NaN) alone, whose exponentials are 0 (or NaN).  +inf leaves NaN.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }
#endif

// Rows that CTAs walk (distill_rows.cu); a cudaError_t as int.
bool distill_walks_rows(const distill_params_t* p);
int launch_distill_rows(const distill_params_t* p, const DistillArgs& A, int mode, cudaStream_t st);

}  // namespace gdn
