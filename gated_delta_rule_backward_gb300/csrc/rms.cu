// rms.cu -- root-mean-square norm with the residual's addition, forward and backward (include/rms.h).
//
// Both directions are one pass over their rows: what is read once is held in registers until
// the row's sums are known.  TPR threads share a row, each with VPT packs of VEC elements, and a
// CTA holds blockDim.y such rows, whose threads meet at a named barrier of their own (a row of one
// warp needs none).  Bytes bound both: a row's loads are all in flight before its first sum.
#include <climits>
#include <cstdio>
#include <cuda_fp8.h>

#include "../../include/rms.h"
#include "gdn_elem.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kMaxThreads = 512;  // of a CTA: 128 registers a thread
constexpr unsigned kAll = 0xffffffffu;
constexpr float kE4m3Max = 448.f;
constexpr float kTinyScale = 1.17549435e-38f;  // 2^-126

struct RmsFwd {
    const void *x, *res, *w;
    void *h, *y;
    float *scales, *rstd;
    long long xs, rs;
    int rows, D, w_dtype, y_dtype, group, vec;
    float eps, inv_D;
};

struct RmsBwd {
    const void *h, *w, *dy, *dh;
    const float* rstd;
    void* dx;
    float* part;  // [gridDim.x][D] sums of dy n over a CTA's rows; null without dweight
    long long hs, dys;
    int rows, D, w_dtype, vec;
    float inv_D;
};

// Sums (and a maximum) over the threads of a row.  buf: two sets of 32 pairs a row of the CTA; successive
// calls alternate between them, so one barrier a call is enough.
__device__ __forceinline__ float2 row_reduce(float s, float m, float2* buf, int tid, int tpr, int bar)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        s += __shfl_xor_sync(kAll, s, o);
        m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    }
    if (tpr > 32) {
        const int lane = tid & 31, warps = tpr >> 5;
        if (lane == 0) buf[tid >> 5] = make_float2(s, m);
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
        const float2 v = lane < warps ? buf[lane] : make_float2(0.f, 0.f);
        s = v.x;
        m = v.y;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            s += __shfl_xor_sync(kAll, s, o);
            m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        }
    }
    return make_float2(s, m);
}

// VEC elements at column c of a row of D (zero past its end).
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> ld_cols(const T* row, int c, int D, bool vec)
{
    Pack<T, VEC> r;
    if (VEC == 1) {
        r.x[0] = c < D ? row[c] : from_f32<T>(0.f);
    } else if (vec) {
        if (c < D) {
            *reinterpret_cast<uint4*>(&r) = *reinterpret_cast<const uint4*>(row + c);
        } else {
            *reinterpret_cast<uint4*>(&r) = make_uint4(0, 0, 0, 0);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.x[i] = c + i < D ? row[c + i] : from_f32<T>(0.f);
    }
    return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void st_cols(T* row, int c, int D, bool vec, const float (&v)[VEC])
{
    if (VEC == 1) {
        if (c < D) row[c] = from_f32<T>(v[0]);
    } else if (vec) {
        constexpr int PER = 16 / (int)sizeof(T);  // elements of one 16-byte store
        if (c < D) {
#pragma unroll
            for (int b = 0; b < VEC; b += PER < VEC ? PER : VEC) {
                Pack<T, PER < VEC ? PER : VEC> r;
#pragma unroll
                for (int i = 0; i < (PER < VEC ? PER : VEC); ++i) r.x[i] = from_f32<T>(v[b + i]);
                if (PER <= VEC) *reinterpret_cast<uint4*>(row + c + b) = *reinterpret_cast<const uint4*>(&r);
                else *reinterpret_cast<uint2*>(row + c + b) = *reinterpret_cast<const uint2*>(&r);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (c + i < D) row[c + i] = from_f32<T>(v[i]);
    }
}

template <int VEC>
__device__ __forceinline__ void ld_weight(float (&w)[VEC], const void* p, int dtype, int c, int D, bool vec)
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] = 1.f;
    } else if (VEC > 1 && vec && c < D && dtype == GDN_F32) {
#pragma unroll
        for (int b = 0; b < VEC; b += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>((const float*)p + c + (VEC > 1 ? b : 0)));
            w[b] = v.x;
            if (VEC > 1) {
                w[b + 1 < VEC ? b + 1 : 0] = v.y;
                w[b + 2 < VEC ? b + 2 : 0] = v.z;
                w[b + 3 < VEC ? b + 3 : 0] = v.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] = c + i < D ? ld_any(p, c + i, dtype) : 0.f;
    }
}

template <int VEC>
__device__ __forceinline__ void st_e4m3(uint8_t* row, int c, int D, bool vec, const float (&v)[VEC])
{
    if (VEC == 1) {
        if (c < D) row[c] = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        uint8_t q[VEC];
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            const __nv_fp8x2_storage_t two =
                __nv_cvt_float2_to_fp8x2(make_float2(v[i], v[VEC > 1 ? i + 1 : 0]), __NV_SATFINITE, __NV_E4M3);
            q[i] = (uint8_t)(two & 0xff);
            q[VEC > 1 ? i + 1 : 0] = (uint8_t)(two >> 8);
        }
        if (vec) {
            if (c < D) {
                uint32_t a = 0;
#pragma unroll
                for (int b = 0; b < VEC; b += 4) {
                    a = 0;
#pragma unroll
                    for (int i = 0; i < 4 && i < VEC; ++i) a |= (uint32_t)q[b + i < VEC ? b + i : 0] << (8 * i);
                    *reinterpret_cast<uint32_t*>(row + c + b) = a;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (c + i < D) row[c + i] = q[i];
        }
    }
}

// h of one pack: x + residual in fp32.
template <typename T, int VEC>
__device__ __forceinline__ void sum_pack(float (&h)[VEC], const Pack<T, VEC>& x, const Pack<T, VEC>& r, bool res)
{
#pragma unroll
    for (int i = 0; i < VEC; ++i) h[i] = res ? x.get(i) + r.get(i) : x.get(i);
}

// What follows the sums, for one pack: h and y (or its codes and scale) to memory.
template <typename T, int VEC>
__device__ __forceinline__ void finish_pack(const RmsFwd& A, const float (&h)[VEC], const float (&w)[VEC], long long row, int c,
                                            float rstd, float inv_scale)
{
    const bool vec = A.vec;
    if (A.h) st_cols<T, VEC>((T*)A.h + row * A.D, c, A.D, vec, h);
    float y[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) y[i] = (h[i] * w[i]) * rstd;
    const long long at = row * A.D;
    if (A.y_dtype == RMS_E4M3) {
        float inv = inv_scale;
        if (VEC > 1 && A.group) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) m = fmaxf(m, fabsf(y[i]));
            const int lanes = A.group / VEC;  // a power of two; every lane of the warp is here
            for (int o = lanes >> 1; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
            const float scale = fmaxf(m / kE4m3Max, kTinyScale);
            inv = 1.f / scale;
            if (c < A.D && (c & (A.group - 1)) == 0) A.scales[row * (A.D / A.group) + c / A.group] = scale;
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) y[i] *= inv;
        st_e4m3<VEC>((uint8_t*)A.y + at, c, A.D, vec, y);
    } else if (A.y_dtype == GDN_F32) {
        st_cols<float, VEC>((float*)A.y + at, c, A.D, vec, y);
    } else if (A.y_dtype == GDN_BF16) {
        st_cols<__nv_bfloat16, VEC>((__nv_bfloat16*)A.y + at, c, A.D, vec, y);
    } else {
        st_cols<__half, VEC>((__half*)A.y + at, c, A.D, vec, y);
    }
}

// VPT packs a thread; VPT = 0: rows that registers do not hold, read again (from L2) after the sums.
template <typename T, int VEC, int VPT>
__global__ void __launch_bounds__(kMaxThreads) rms_forward_kernel(const RmsFwd A)
{
    __shared__ float2 buf[32 * 16];
    const int tid = threadIdx.x, tpr = blockDim.x;
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= A.rows) return;  // the whole row's threads leave together
    const T* x = (const T*)A.x + row * A.xs;
    const T* r = A.res ? (const T*)A.res + row * A.rs : x;
    const bool res = A.res != nullptr;
    float s = 0.f, m = 0.f;
    float h[VPT ? VPT : 1][VEC], w[VPT ? VPT : 1][VEC];
    const int step = tpr * VEC;
    if (VPT) {
        Pack<T, VEC> px[VPT ? VPT : 1], pr[VPT ? VPT : 1];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            px[v] = ld_cols<T, VEC>(x, tid * VEC + v * step, A.D, A.vec);
            if (res) pr[v] = ld_cols<T, VEC>(r, tid * VEC + v * step, A.D, A.vec);
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) ld_weight<VEC>(w[v], A.w, A.w_dtype, tid * VEC + v * step, A.D, A.vec);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            sum_pack<T, VEC>(h[v], px[v], pr[v], res);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s = fmaf(h[v][i], h[v][i], s);
                m = fmaxf(m, fabsf(h[v][i] * w[v][i]));
            }
        }
    } else {
        for (int c = tid * VEC; c < A.D; c += step) {
            const Pack<T, VEC> px = ld_cols<T, VEC>(x, c, A.D, A.vec), pr = ld_cols<T, VEC>(r, c, A.D, A.vec);
            sum_pack<T, VEC>(h[0], px, pr, res);
            ld_weight<VEC>(w[0], A.w, A.w_dtype, c, A.D, A.vec);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s = fmaf(h[0][i], h[0][i], s);
                m = fmaxf(m, fabsf(h[0][i] * w[0][i]));
            }
        }
    }
    const float2 sm = row_reduce(s, m, buf + 32 * threadIdx.y, tid, tpr, 1 + threadIdx.y);
    const float rstd = 1.f / sqrtf(sm.x * A.inv_D + A.eps);
    const float scale = fmaxf(sm.y * rstd / kE4m3Max, kTinyScale), inv = 1.f / scale;
    if (tid == 0) {
        if (A.rstd) A.rstd[row] = rstd;
        if (A.y_dtype == RMS_E4M3 && !A.group) A.scales[row] = scale;
    }
    if (VPT) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) finish_pack<T, VEC>(A, h[v], w[v], row, tid * VEC + v * step, rstd, inv);
    } else {
        // whole steps, so that the lanes that share a scale stay together
        for (int c0 = 0; c0 < A.D; c0 += step) {
            const int c = c0 + tid * VEC;
            const Pack<T, VEC> px = ld_cols<T, VEC>(x, c, A.D, A.vec), pr = ld_cols<T, VEC>(r, c, A.D, A.vec);
            sum_pack<T, VEC>(h[0], px, pr, res);
            ld_weight<VEC>(w[0], A.w, A.w_dtype, c, A.D, A.vec);
            finish_pack<T, VEC>(A, h[0], w[0], row, c, rstd, inv);
        }
    }
}

// Rows blockIdx.x blockDim.y + threadIdx.y, then a whole grid of rows further: a thread keeps its columns,
// their weights and their part of dweight in registers over all its rows.
template <typename T, int VEC, int VPT>
__global__ void __launch_bounds__(kMaxThreads) rms_backward_kernel(const RmsBwd A)
{
    extern __shared__ float sums[];  // [blockDim.y][D] at the end
    __shared__ float2 buf[2][32 * 16];
    const int tid = threadIdx.x, tpr = blockDim.x, step = tpr * VEC;
    float w[VPT][VEC], dw[VPT][VEC];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        ld_weight<VEC>(w[v], A.w, A.w_dtype, tid * VEC + v * step, A.D, A.vec);
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[v][i] = 0.f;
    }
    int set = 0;
    for (long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y; row < A.rows;
         row += (long long)gridDim.x * blockDim.y, set ^= 1) {
        const T *h = (const T*)A.h + row * A.hs, *dy = (const T*)A.dy + row * A.dys;
        const T* dh = A.dh ? (const T*)A.dh + row * A.D : nullptr;
        const float rstd = __ldg(A.rstd + row);
        Pack<T, VEC> ph[VPT], pd[VPT], pg[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = tid * VEC + v * step;
            ph[v] = ld_cols<T, VEC>(h, c, A.D, A.vec);
            pd[v] = ld_cols<T, VEC>(dy, c, A.D, A.vec);
            if (dh) pg[v] = ld_cols<T, VEC>(dh, c, A.D, A.vec);
        }
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float n = ph[v].get(i) * rstd, d = pd[v].get(i);
                s = fmaf(d * w[v][i], n, s);
                dw[v][i] = fmaf(d, n, dw[v][i]);
            }
        const float c = row_reduce(s, 0.f, buf[set] + 32 * threadIdx.y, tid, tpr, 1 + threadIdx.y).x * A.inv_D;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                o[i] = rstd * fmaf(-(ph[v].get(i) * rstd), c, pd[v].get(i) * w[v][i]);
                if (dh) o[i] += pg[v].get(i);
            }
            st_cols<T, VEC>((T*)A.dx + row * A.D, tid * VEC + v * step, A.D, A.vec, o);
        }
    }
    if (!A.part) return;
    float* mine = sums + (size_t)threadIdx.y * A.D;
    float* out = A.part + (size_t)blockIdx.x * A.D;
    if (blockDim.y > 1) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int c = tid * VEC + v * step + i;
                if (c < A.D) mine[c] = dw[v][i];
            }
        __syncthreads();
        for (int c = threadIdx.y * tpr + tid; c < A.D; c += tpr * blockDim.y) {
            float t = 0.f;
            for (int r = 0; r < (int)blockDim.y; ++r) t += sums[(size_t)r * A.D + c];
            out[c] = t;
        }
    } else {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int c = tid * VEC + v * step + i;
                if (c < A.D) out[c] = dw[v][i];
            }
    }
}

// Rows that registers do not hold: dx row by row, read twice; dweight's parts by the kernel below.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) rms_backward_long_kernel(const RmsBwd A)
{
    __shared__ float2 buf[32];
    const long long row = blockIdx.x;
    const T *h = (const T*)A.h + row * A.hs, *dy = (const T*)A.dy + row * A.dys;
    const T* dh = A.dh ? (const T*)A.dh + row * A.D : nullptr;
    const float rstd = __ldg(A.rstd + row);
    float s = 0.f;
    for (int c = threadIdx.x; c < A.D; c += blockDim.x)
        s = fmaf(to_f32(dy[c]) * (A.w ? ld_any(A.w, c, A.w_dtype) : 1.f), to_f32(h[c]) * rstd, s);
    const float m = row_reduce(s, 0.f, buf, threadIdx.x, blockDim.x, 1).x * A.inv_D;
    for (int c = threadIdx.x; c < A.D; c += blockDim.x) {
        float o = rstd * fmaf(-(to_f32(h[c]) * rstd), m, to_f32(dy[c]) * (A.w ? ld_any(A.w, c, A.w_dtype) : 1.f));
        if (dh) o += to_f32(dh[c]);
        ((T*)A.dx)[row * A.D + c] = from_f32<T>(o);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) rms_dweight_long_kernel(const RmsBwd A)
{
    const int c = blockIdx.y * 256 + threadIdx.x;
    if (c >= A.D) return;
    float t = 0.f;
    for (long long row = blockIdx.x; row < A.rows; row += gridDim.x)
        t = fmaf(to_f32(((const T*)A.dy)[row * A.dys + c]), to_f32(((const T*)A.h)[row * A.hs + c]) * __ldg(A.rstd + row), t);
    A.part[(size_t)blockIdx.x * A.D + c] = t;
}

// dweight = the parts' sum, 32 columns a CTA, 8 warps over the parts.
__global__ void __launch_bounds__(256) rms_dweight_sum_kernel(const float* part, int parts, int D, float* dweight)
{
    __shared__ float s[8][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    float t = 0.f;
    if (c < D)
        for (int p = g; p < parts; p += 8) t += part[(size_t)p * D + c];
    s[g][threadIdx.x & 31] = t;
    __syncthreads();
    if (g == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) t += s[i][threadIdx.x];
        dweight[c] = t;
    }
}

// How a row is laid over threads: tpr threads of vpt packs (0: more than registers hold), ry rows a CTA.
struct Shape {
    int vec, vpt, tpr, ry;
};

// The layout, and with it the order of every sum, goes by D, the rows and the types alone: the same numbers give the
// same bits whatever their alignment (packs off their 16 bytes are loaded one by one).
Shape shape_of(const rms_params_t* p, int max_regs)
{
    const int64_t D = p->D, rows = p->rows;
    const int vecn = 16 / (int)elem_size(p->x_dtype);
    Shape s{};
    s.vec = D % vecn == 0 ? vecn : 1;
    const int64_t packs = (D + s.vec - 1) / s.vec;
    const int most = max_regs / s.vec;  // packs that a thread's registers hold
    s.vpt = 1;
    while (s.vpt < most && packs > 256 * (int64_t)s.vpt) s.vpt *= 2;
    int64_t t = (packs + s.vpt - 1) / s.vpt;
    t = (t + 31) / 32 * 32;
    if (t > kMaxThreads) {
        s.vpt = 0;
        t = kMaxThreads;
    }
    s.tpr = (int)t;
    s.ry = s.tpr >= 256 ? 1 : 256 / s.tpr;
    while (s.ry > 1 && rows < (int64_t)s.ry * kNumSMs) s.ry /= 2;
    return s;
}

template <typename T, int VEC>
int launch_fwd(const RmsFwd& A, const Shape& s, cudaStream_t st)
{
    const dim3 block(s.tpr, s.ry);
    const unsigned grid = (unsigned)((A.rows + s.ry - 1) / s.ry);
    constexpr int M = 32 / VEC;  // most packs of a thread
    if (s.vpt == 0) rms_forward_kernel<T, VEC, 0><<<grid, block, 0, st>>>(A);
    else if (s.vpt == 1) rms_forward_kernel<T, VEC, 1><<<grid, block, 0, st>>>(A);
    else if (s.vpt == 2) rms_forward_kernel<T, VEC, 2><<<grid, block, 0, st>>>(A);
    else if (s.vpt == 4) rms_forward_kernel<T, VEC, 4><<<grid, block, 0, st>>>(A);
    else if (s.vpt == 8) rms_forward_kernel<T, VEC, M < 8 ? M : 8><<<grid, block, 0, st>>>(A);
    else if (s.vpt == 16) rms_forward_kernel<T, VEC, M < 16 ? M : 16><<<grid, block, 0, st>>>(A);
    else rms_forward_kernel<T, VEC, M><<<grid, block, 0, st>>>(A);
    return (int)cudaGetLastError();
}

template <typename T, int VEC, int VPT>
int launch_bwd_v(const RmsBwd& A, const Shape& s, int ctas, cudaStream_t st)
{
    const size_t smem = A.part && s.ry > 1 ? (size_t)s.ry * A.D * 4 : 0;
    if (smem > 40 * 1024) {
        const int e = (int)cudaFuncSetAttribute(rms_backward_kernel<T, VEC, VPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e) return e;
    }
    rms_backward_kernel<T, VEC, VPT><<<ctas, dim3(s.tpr, s.ry), smem, st>>>(A);
    return (int)cudaGetLastError();
}

template <typename T, int VEC>
int launch_bwd(const RmsBwd& A, const Shape& s, int ctas, cudaStream_t st)
{
    constexpr int M = 16 / VEC < 1 ? 1 : 16 / VEC;
    if (s.vpt == 0) {
        rms_backward_long_kernel<T><<<(unsigned)A.rows, kMaxThreads, 0, st>>>(A);
        if (A.part) rms_dweight_long_kernel<T><<<dim3(ctas, (A.D + 255) / 256), 256, 0, st>>>(A);
        return (int)cudaGetLastError();
    }
    if (s.vpt == 1) return launch_bwd_v<T, VEC, 1>(A, s, ctas, st);
    if (s.vpt == 2) return launch_bwd_v<T, VEC, 2>(A, s, ctas, st);
    if (s.vpt == 4) return launch_bwd_v<T, VEC, M < 4 ? M : 4>(A, s, ctas, st);
    if (s.vpt == 8) return launch_bwd_v<T, VEC, M < 8 ? M : 8>(A, s, ctas, st);
    return launch_bwd_v<T, VEC, M>(A, s, ctas, st);
}

// CTAs of the backward, each with its own part of dweight: every SM's registers once.
int bwd_ctas(const rms_params_t* p, const Shape& s)
{
    int64_t per_sm = 1024 / (s.tpr * s.ry);
    if (per_sm < 1) per_sm = 1;
    const int64_t need = (p->rows + s.ry - 1) / s.ry;
    return (int)(need < kNumSMs * per_sm ? need : kNumSMs * per_sm);
}

int fail(int code, const char* msg)
{
    set_last_error(msg);
    return code;
}

int cuda_fail(int e, const char* what)
{
    char msg[256];
    snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString((cudaError_t)e));
    return fail(GDN_ERR_CUDA, msg);
}

bool overlap(const void* a, size_t na, const void* b, size_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && na && nb && x < y + nb && y < x + na;
}

int check(const rms_params_t* p)
{
    if (!p) return fail(GDN_ERR_INVALID_ARG, "rms: params is NULL");
    if (p->rows < 0 || p->D < 1) return fail(GDN_ERR_INVALID_ARG, "rms: rows must be >= 0 and D >= 1");
    if (p->x_s < p->D || p->res_s < p->D) return fail(GDN_ERR_INVALID_ARG, "rms: a row stride is below D");
    if (!known_dtype(p->x_dtype) || !known_dtype(p->w_dtype) || !(known_dtype(p->y_dtype) || p->y_dtype == RMS_E4M3))
        return fail(GDN_ERR_INVALID_ARG, "rms: unknown dtype");
    if (p->group != 0 && p->group != 16 && p->group != 32 && p->group != 64 && p->group != 128)
        return fail(GDN_ERR_UNSUPPORTED, "rms: group must be 0, 16, 32, 64 or 128");
    if (p->group && p->D % p->group != 0) return fail(GDN_ERR_INVALID_ARG, "rms: group does not divide D");
    if (p->rows > INT_MAX || p->D > (1 << 28)) return fail(GDN_ERR_UNSUPPORTED, "rms: sizes beyond the kernels' index range");
    return GDN_OK;
}

bool wide_ok(const rms_params_t* p, std::initializer_list<const void*> ptrs)
{
    const int vecn = 16 / (int)elem_size(p->x_dtype);
    for (const void* q : ptrs)
        if ((uintptr_t)q % 16 != 0) return false;
    return p->D % vecn == 0 && p->x_s % vecn == 0 && p->res_s % vecn == 0;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" size_t rms_backward_workspace_bytes(const rms_params_t* p)
{
    if (check(p) != GDN_OK || p->rows == 0) return 0;
    return (size_t)bwd_ctas(p, shape_of(p, 16)) * p->D * 4;
}

extern "C" int rms_forward(const rms_params_t* p, const void* x, const void* residual, const void* weight, void* h, void* y,
                           float* scales, float* rstd, void* stream)
{
    const int st = check(p);
    if (st != GDN_OK) return st;
    if (p->rows == 0) return GDN_OK;
    const bool e4 = p->y_dtype == RMS_E4M3;
    if (!x || !y || (e4 && !scales)) return fail(GDN_ERR_INVALID_ARG, "rms_forward: NULL pointer");
    const size_t es = elem_size(p->x_dtype), ws = elem_size(p->w_dtype), ys = e4 ? 1 : elem_size(p->y_dtype);
    if ((uintptr_t)x % es || (uintptr_t)residual % es || (uintptr_t)h % es || (uintptr_t)weight % ws || (uintptr_t)y % ys ||
        (uintptr_t)scales % 4 || (uintptr_t)rstd % 4)
        return fail(GDN_ERR_INVALID_ARG, "rms_forward: a pointer is not aligned to its element");
    const size_t n = (size_t)(p->rows * p->D);
    const size_t n_x = (size_t)((p->rows - 1) * p->x_s + p->D) * es, n_r = residual ? (size_t)((p->rows - 1) * p->res_s + p->D) * es : 0;
    const size_t n_sc = e4 ? (size_t)p->rows * (p->group ? p->D / p->group : 1) * 4 : 0;
    const struct { const void* ptr; size_t n; } out[] = {{h, n * es}, {y, n * ys}, {scales, n_sc}, {rstd, (size_t)p->rows * 4}};
    for (int i = 0; i < 4; ++i) {
        const bool in_place_x = i == 0 && h == x && p->x_s == p->D, in_place_r = i == 0 && h == residual && p->res_s == p->D;
        if ((!in_place_x && overlap(out[i].ptr, out[i].n, x, n_x)) || (!in_place_r && overlap(out[i].ptr, out[i].n, residual, n_r)) ||
            overlap(out[i].ptr, out[i].n, weight, (size_t)p->D * ws))
            return fail(GDN_ERR_ALIAS, "rms_forward: an output overlaps an input");
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].ptr, out[i].n, out[j].ptr, out[j].n)) return fail(GDN_ERR_ALIAS, "rms_forward: outputs overlap");
    }
    RmsFwd A{};
    A.x = x; A.res = residual; A.w = weight; A.h = h; A.y = y; A.scales = e4 ? scales : nullptr; A.rstd = rstd;
    A.xs = p->x_s; A.rs = p->res_s; A.rows = (int)p->rows; A.D = (int)p->D;
    A.w_dtype = p->w_dtype; A.y_dtype = p->y_dtype; A.group = e4 ? p->group : 0;
    A.eps = p->eps; A.inv_D = 1.f / (float)p->D;
    A.vec = wide_ok(p, {x, residual, weight, h, y});
    const Shape s = shape_of(p, 32);
    cudaStream_t cs = (cudaStream_t)stream;
    int e;
    if (p->x_dtype == GDN_F32) e = s.vec > 1 ? launch_fwd<float, 4>(A, s, cs) : launch_fwd<float, 1>(A, s, cs);
    else if (p->x_dtype == GDN_BF16) e = s.vec > 1 ? launch_fwd<__nv_bfloat16, 8>(A, s, cs) : launch_fwd<__nv_bfloat16, 1>(A, s, cs);
    else e = s.vec > 1 ? launch_fwd<__half, 8>(A, s, cs) : launch_fwd<__half, 1>(A, s, cs);
    return e ? cuda_fail(e, "rms_forward launch") : GDN_OK;
}

extern "C" int rms_backward(const rms_params_t* p, const void* h, const void* weight, const float* rstd, const void* dy,
                            const void* dh, void* dx, float* dweight, void* workspace, size_t workspace_bytes, void* stream)
{
    const int st = check(p);
    if (st != GDN_OK) return st;
    cudaStream_t cs = (cudaStream_t)stream;
    if (p->rows == 0) {
        if (!dweight) return GDN_OK;
        const int e = (int)cudaMemsetAsync(dweight, 0, (size_t)p->D * 4, cs);
        return e ? cuda_fail(e, "rms_backward") : GDN_OK;
    }
    if (!h || !rstd || !dy || !dx) return fail(GDN_ERR_INVALID_ARG, "rms_backward: NULL pointer");
    const size_t es = elem_size(p->x_dtype), ws = elem_size(p->w_dtype);
    if ((uintptr_t)h % es || (uintptr_t)dy % es || (uintptr_t)dh % es || (uintptr_t)dx % es || (uintptr_t)weight % ws ||
        (uintptr_t)rstd % 4 || (uintptr_t)dweight % 4 || (uintptr_t)workspace % 16)
        return fail(GDN_ERR_INVALID_ARG, "rms_backward: a pointer is not aligned to its element (the workspace to 16 bytes)");
    const size_t need = rms_backward_workspace_bytes(p);
    if (dweight && (!workspace || workspace_bytes < need))
        return fail(GDN_ERR_WORKSPACE, "rms_backward: workspace smaller than rms_backward_workspace_bytes()");
    const size_t n = (size_t)(p->rows * p->D) * es;
    const struct { const void* ptr; size_t n; } in[] = {
        {h, (size_t)((p->rows - 1) * p->x_s + p->D) * es}, {dy, (size_t)((p->rows - 1) * p->res_s + p->D) * es}, {dh, n},
        {weight, (size_t)p->D * ws}, {rstd, (size_t)p->rows * 4}};
    const struct { const void* ptr; size_t n; } out[] = {{dx, n}, {dweight, (size_t)p->D * 4}, {dweight ? workspace : nullptr, need}};
    for (int i = 0; i < 3; ++i) {
        for (const auto& o : in)
            if (overlap(out[i].ptr, out[i].n, o.ptr, o.n)) return fail(GDN_ERR_ALIAS, "rms_backward: an output overlaps an input");
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].ptr, out[i].n, out[j].ptr, out[j].n)) return fail(GDN_ERR_ALIAS, "rms_backward: outputs overlap");
    }
    RmsBwd A{};
    A.h = h; A.w = weight; A.dy = dy; A.dh = dh; A.rstd = rstd; A.dx = dx; A.part = dweight ? (float*)workspace : nullptr;
    A.hs = p->x_s; A.dys = p->res_s; A.rows = (int)p->rows; A.D = (int)p->D; A.w_dtype = p->w_dtype;
    A.inv_D = 1.f / (float)p->D;
    A.vec = wide_ok(p, {h, weight, dy, dh, dx});
    const Shape s = shape_of(p, 16);
    const int ctas = bwd_ctas(p, s);
    int e;
    if (p->x_dtype == GDN_F32) e = s.vec > 1 ? launch_bwd<float, 4>(A, s, ctas, cs) : launch_bwd<float, 1>(A, s, ctas, cs);
    else if (p->x_dtype == GDN_BF16) e = s.vec > 1 ? launch_bwd<__nv_bfloat16, 8>(A, s, ctas, cs) : launch_bwd<__nv_bfloat16, 1>(A, s, ctas, cs);
    else e = s.vec > 1 ? launch_bwd<__half, 8>(A, s, ctas, cs) : launch_bwd<__half, 1>(A, s, ctas, cs);
    if (!e && dweight) {
        rms_dweight_sum_kernel<<<(unsigned)((p->D + 31) / 32), 256, 0, cs>>>(A.part, ctas, A.D, dweight);
        e = (int)cudaGetLastError();
    }
    return e ? cuda_fail(e, "rms_backward launch") : GDN_OK;
}
