// rms.cu -- root-mean-square norm with the residual's addition, forward and backward (include/rms.h).
//
// Both directions are one pass over their rows: what is read once is held in registers until the
// row's sums are known.  TPR threads share a row, each with VPT packs of VEC elements (16 bytes), two to
// a register pair for the packed fp32 instructions.  Bytes bound both.
//
// Packs lie at multiples of VEC of the flat index row D + column, so that they are aligned for any D: where VEC does
// not divide D, a row begins `lead` elements into its first pack and may end inside its last.  A cut pack is still
// read as a whole (its other elements are a neighbouring row's, and set to zero) and stored one by one.
//
// Forward: a CTA a row (a warp where rows are short), five CTAs an SM, so that other rows' loads
// are in flight while one is summed; with y = (h w) rstd the largest |h w| of a row, summed beside
// the squares, gives its scale without a second exchange.  Measured: 4096 rows of 6144, bf16 to codes with a
// scale for 128 columns, 30.0 us, 5.9 TB/s of 6.7 for a copy; 4096 of 4095 bf16 30.7 us,
// 4.4 TB/s; one row of 2048 1.9 us (in a graph).
// Backward: one persistent CTA of 512 threads an SM, 16 elements a thread (a row's exchange costs
// about as much as 16 elements' arithmetic), rows through a ring of asynchronous copies, dweight
// in registers over all rows, then one part a CTA and a second kernel that sums 152 parts.
// Measured: 8192 rows of 2048, bf16, 28.2 us in all; 4096 of 4095 39 us.
#include <climits>
#include <cstdio>
#include <cuda_fp8.h>

#include "../../include/rms.h"
#include "gdn_elem.cuh"
#include "gdn_f32x2.cuh"
#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_packs.h"

namespace gdn {
namespace {

constexpr int kMaxThreads = 1024, kRingThreads = 512;
constexpr int kMostSmem = 220 * 1024;  // of a backward CTA, beside its static arrays
constexpr unsigned kAll = 0xffffffffu;
constexpr float kE4m3Max = 448.f;
constexpr float kTinyScale = 1.17549435e-38f;  // 2^-126

struct RmsFwd {
    const void *x, *res, *w;
    void *h, *y;
    float *scales, *rstd;
    long long xs, rs;
    int rows, D, w_dtype, y_dtype, lg_group, vec, w_vec;
    float eps, inv_D;
};

struct RmsBwd {
    const void *h, *w, *dy, *dh;
    const float* rstd;
    void* dx;
    float* part;  // [gridDim.x][D] sums of dy n over a CTA's rows; null without dweight
    long long hs, dys;
    int rows, D, w_dtype, vec, w_vec;
    float inv_D;
};

// A sum (MAX: a maximum too) over the threads of a row: a warp, a CTA, or (GROUPS) one of several rows of a CTA,
// which meet at a named barrier of their own.  buf: 32 pairs for each row; successive calls use different
// ones, so one barrier a call is enough.
template <bool MAX, bool GROUPS>
__device__ __forceinline__ float2 row_reduce(float s, float m, float2* buf)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        s += __shfl_xor_sync(kAll, s, o);
        if (MAX) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    }
    if (blockDim.x > 32) {
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float2(s, m);
        if (GROUPS) asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.y), "r"(blockDim.x) : "memory");
        else __syncthreads();
        s = m = 0.f;
        for (int i = 0; i < (int)(blockDim.x >> 5); ++i) {
            const float2 v = buf[i];
            s += v.x;
            if (MAX) m = fmaxf(m, v.y);
        }
    }
    return make_float2(s, m);
}

// VEC fp32 numbers, in pairs for the packed fp32 pipe.
template <int VEC>
struct Nums {
    f2 v[VEC / 2];
    __device__ __forceinline__ void fill(float x)
    {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) v[i] = pack2(x, x);
    }
    __device__ __forceinline__ void set(int i, float x, float y) { v[i / 2] = pack2(x, y); }
    __device__ __forceinline__ float2 pair(int i) const { return unpack2(v[i / 2]); }
    __device__ __forceinline__ float sum() const
    {
        f2 t = v[0];
#pragma unroll
        for (int i = 1; i < VEC / 2; ++i) t = add2(t, v[i]);
        return sum2(t);
    }
    __device__ __forceinline__ float max_abs() const
    {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const float2 x = unpack2(v[i]);
            m = fmaxf(m, fmaxf(fabsf(x.x), fabsf(x.y)));
        }
        return m;
    }
};
template <int VEC>
__device__ __forceinline__ Nums<VEC> add(const Nums<VEC>& a, const Nums<VEC>& b)
{
    Nums<VEC> r;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) r.v[i] = add2(a.v[i], b.v[i]);
    return r;
}
template <int VEC>
__device__ __forceinline__ Nums<VEC> mul(const Nums<VEC>& a, const Nums<VEC>& b)
{
    Nums<VEC> r;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) r.v[i] = mul2(a.v[i], b.v[i]);
    return r;
}
template <int VEC>
__device__ __forceinline__ Nums<VEC> mul(const Nums<VEC>& a, float b)
{
    Nums<VEC> r;
    const f2 bb = pack2(b, b);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) r.v[i] = mul2(a.v[i], bb);
    return r;
}
template <int VEC>
__device__ __forceinline__ Nums<VEC> fma(const Nums<VEC>& a, const Nums<VEC>& b, const Nums<VEC>& c)
{
    Nums<VEC> r;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) r.v[i] = fma2(a.v[i], b.v[i], c.v[i]);
    return r;
}
template <int VEC>
__device__ __forceinline__ Nums<VEC> fma(const Nums<VEC>& a, float b, const Nums<VEC>& c)
{
    Nums<VEC> r;
    const f2 bb = pack2(b, b);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) r.v[i] = fma2(a.v[i], bb, c.v[i]);
    return r;
}

__device__ __forceinline__ float2 widen2(uint32_t w, __nv_bfloat16) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ float2 widen2(uint32_t w, __half) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ uint32_t narrow2(float2 x, __nv_bfloat16)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t narrow2(float2 x, __half)
{
    const __half2 v = __floats2half2_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// The first `from` and the elements past `to` of a pack set to zero.
template <typename T>
__device__ __forceinline__ uint4 cut_pack(const uint4& x, int from, int to)
{
    constexpr int PER = 4 / (int)sizeof(T);  // elements of a word
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4 * PER; ++i)
        if (i < from || i >= to) w[i / PER] &= PER == 1 ? 0u : i & 1 ? 0xffffu : 0xffff0000u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// How a tensor's packs are reached: whole and aligned, aligned but cut by the rows' ends, or element by element.
enum { kWhole = 0, kCut = 1, kSingle = 2 };

// The pack at column c of a row of D (zero outside the row), as it is stored.  `more`: what lies around the row in memory
// may be read, too.
template <typename T, int VEC, int HOW>
__device__ __forceinline__ uint4 ld_cols(const T* row, int c, int D, bool more)
{
    uint4 r = make_uint4(0, 0, 0, 0);
    if (HOW == kWhole) {
        if (c < D) r = *reinterpret_cast<const uint4*>(row + c);
        return r;
    }
    const bool whole = c >= 0 && c + VEC <= D;
    if (HOW == kCut) {
        if (c < D && (whole || more)) r = *reinterpret_cast<const uint4*>(row + c);
        if (whole || c >= D) return r;
        if (more) return cut_pack<T>(r, -c, D - c);
    }
    if (c < D) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (c + i >= 0 && c + i < D) {
                if (sizeof(T) == 4) w[i & 3] = reinterpret_cast<const uint32_t*>(row)[c + i];
                else w[(i / 2) & 3] |= (uint32_t) reinterpret_cast<const uint16_t*>(row)[c + i] << (16 * (i & 1));
            }
        r = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return r;
}

template <typename T, int VEC>
__device__ __forceinline__ Nums<VEC> widen(const uint4& x)
{
    Nums<VEC> r;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) r.set(i, __uint_as_float(w[i]), __uint_as_float(w[i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const float2 v = widen2(w[i], T());
            r.set(2 * i, v.x, v.y);
        }
    }
    return r;
}

template <typename T, int VEC, int HOW>
__device__ __forceinline__ void st_cols(T* row, int c, int D, const Nums<VEC>& v)
{
    if (HOW == kWhole || (HOW == kCut && c >= 0 && c + VEC <= D)) {
        if (HOW == kWhole && c >= D) return;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VEC; i += 4) {
                const float2 a = v.pair(i), b = v.pair(i + 2);
                *reinterpret_cast<float4*>(row + c + i) = make_float4(a.x, a.y, b.x, b.y);
            }
        } else if constexpr (VEC == 8) {
            *reinterpret_cast<uint4*>(row + c) = make_uint4(narrow2(v.pair(0), T()), narrow2(v.pair(2), T()), narrow2(v.pair(4), T()), narrow2(v.pair(6), T()));
        } else {
            *reinterpret_cast<uint2*>(row + c) = make_uint2(narrow2(v.pair(0), T()), narrow2(v.pair(2), T()));
        }
    } else if (c < D) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            const float2 a = v.pair(i);
            if (c + i >= 0 && c + i < D) row[c + i] = from_f32<T>(a.x);
            if (c + i + 1 >= 0 && c + i + 1 < D) row[c + i + 1] = from_f32<T>(a.y);
        }
    }
}

template <int VEC, int HOW>
__device__ __forceinline__ Nums<VEC> ld_weight(const void* p, int dtype, int c, int D, bool vec)
{
    Nums<VEC> w;
    if (!p) {
        w.fill(1.f);
    } else if (HOW == kWhole && vec && dtype == GDN_F32) {
#pragma unroll
        for (int b = 0; b < VEC; b += 4) {
            const float4 v = c < D ? ld_plain(reinterpret_cast<const float4*>((const float*)p + c + b)) : make_float4(0.f, 0.f, 0.f, 0.f);
            w.set(b, v.x, v.y);
            w.set(b + 2, v.z, v.w);
        }
    } else if (HOW == kCut && vec && dtype == GDN_F32 && c >= 0 && (c & ~3) + VEC + 4 <= D) {
        // c is not a multiple of 4: the 16-byte loads around it, moved on by c mod 4 (the same for the whole row)
        const float* q = (const float*)p + (c & ~3);
        float x[VEC + 4];
#pragma unroll
        for (int b = 0; b < VEC + 4; b += 4) {
            const float4 v = ld_plain(reinterpret_cast<const float4*>(q + b));
            x[b] = v.x;
            x[b + 1] = v.y;
            x[b + 2] = v.z;
            x[b + 3] = v.w;
        }
        const bool one = c & 1, two = c & 2;
#pragma unroll
        for (int i = 0; i < VEC + 2; ++i) x[i] = one ? x[i + 1] : x[i];
#pragma unroll
        for (int i = 0; i < VEC; i += 2) w.set(i, two ? x[i + 2] : x[i], two ? x[i + 3] : x[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2)
            w.set(i, c + i >= 0 && c + i < D ? ld_any(p, c + i, dtype) : 0.f, c + i + 1 >= 0 && c + i + 1 < D ? ld_any(p, c + i + 1, dtype) : 0.f);
    }
    return w;
}

template <int VEC, int HOW>
__device__ __forceinline__ void st_e4m3(uint8_t* row, int c, int D, const Nums<VEC>& v)
{
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(v.pair(i), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(v.pair(i + 2), __NV_SATFINITE, __NV_E4M3);
        w[i / 4] = lo | hi << 16;
    }
    if (HOW == kWhole || (HOW == kCut && c >= 0 && c + VEC <= D)) {
        if (HOW == kWhole && c >= D) return;
        if constexpr (VEC == 8) *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(row + c) = w[0];
    } else if (c < D) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (c + i >= 0 && c + i < D) row[c + i] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
    }
}

// The forms of y: a type of its own, 8-bit codes with a scale a row, or a scale a group of columns.
enum { kPlain = 0, kRowCodes = 1, kGroupCodes = 2 };

// What follows the sums, for one pack: h and y (or its codes and scale) to memory.
template <typename T, int VEC, int OUT, int HOW>
__device__ __forceinline__ void finish_pack(const RmsFwd& A, const Nums<VEC>& h, long long row, int c, float rstd, float inv)
{
    const long long at = row * A.D;
    if (A.h) st_cols<T, VEC, HOW>((T*)A.h + at, c, A.D, h);
    const Nums<VEC> y = mul(mul(h, ld_weight<VEC, HOW>(A.w, A.w_dtype, c, A.D, A.w_vec)), rstd);
    if (OUT == kGroupCodes) {
        float m = y.max_abs();
        // the lanes of a group (a power of two; every lane of the warp is here)
        if (A.lg_group == 7) {
#pragma unroll
            for (int o = 64 / VEC; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        } else {
            for (int o = (1 << A.lg_group) / VEC / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        }
        const float scale = fmaxf(m * (1.f / kE4m3Max), kTinyScale);
        inv = __frcp_rn(scale);
        if (c < A.D && (c & ((1 << A.lg_group) - 1)) == 0) A.scales[row * (A.D >> A.lg_group) + (c >> A.lg_group)] = scale;
    }
    if (OUT != kPlain) {
        st_e4m3<VEC, HOW>((uint8_t*)A.y + at, c, A.D, mul(y, inv));
    } else if (A.y_dtype == GDN_BF16) {
        st_cols<__nv_bfloat16, VEC, HOW>((__nv_bfloat16*)A.y + at, c, A.D, y);
    } else if (A.y_dtype == GDN_F32) {
        st_cols<float, VEC, HOW>((float*)A.y + at, c, A.D, y);
    } else {
        st_cols<__half, VEC, HOW>((__half*)A.y + at, c, A.D, y);
    }
}

// VPT packs a thread; VPT = 0: rows that registers do not hold, read again (from L2) after the sums.
// Rows of fewer than the most packs have 256 threads at most, five CTAs an SM: 4096 rows of 6144 to codes take
// 29.5 us so in a graph (a scale a row: 31.3), 30.5 us (34.0) with the compiler's own choice of registers.
template <typename T, int VPT, int OUT, int HOW>
__global__ void __launch_bounds__(VPT > 0 && VPT < 4 ? 256 : kMaxThreads, VPT > 0 && VPT < 4 ? (HOW == kWhole ? 5 : 4) : 1) rms_forward_kernel(const RmsFwd A)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    __shared__ float2 buf[32];
    const int tid = threadIdx.x, step = blockDim.x * VEC;
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    begin_after();
    if (row >= A.rows) return;  // the whole row's threads leave together
    const int c0 = tid * VEC - (HOW != kWhole ? pack_lead(row, A.D, VEC) : 0);
    const T* x = (const T*)A.x + row * A.xs;
    const T* r = A.res ? (const T*)A.res + row * A.rs : x;
    // a sum that replaces an input row may only be read by its own row's threads
    const bool more = HOW == kCut && row + 1 < A.rows && A.h != A.x && A.h != A.res;
    Nums<VEC> h[VPT ? VPT : 1], acc;
    acc.fill(0.f);
    float m = 0.f;
    auto sum_at = [&](int c) {
        const uint4 a = ld_cols<T, VEC, HOW>(x, c, A.D, more);
        if (!A.res) return widen<T, VEC>(a);
        return add(widen<T, VEC>(a), widen<T, VEC>(ld_cols<T, VEC, HOW>(r, c, A.D, more)));
    };
    auto take = [&](const Nums<VEC>& hv, int c) {
        acc = fma(hv, hv, acc);
        if (OUT == kRowCodes) m = fmaxf(m, mul(hv, ld_weight<VEC, HOW>(A.w, A.w_dtype, c, A.D, A.w_vec)).max_abs());
    };
    if (VPT) {
        uint4 px[VPT ? VPT : 1], pr[VPT ? VPT : 1];
#pragma unroll
        for (int v = 0; v < VPT; ++v) px[v] = ld_cols<T, VEC, HOW>(x, c0 + v * step, A.D, more);
        if (A.res) {
#pragma unroll
            for (int v = 0; v < VPT; ++v) pr[v] = ld_cols<T, VEC, HOW>(r, c0 + v * step, A.D, more);
#pragma unroll
            for (int v = 0; v < VPT; ++v) h[v] = add(widen<T, VEC>(px[v]), widen<T, VEC>(pr[v]));
        } else {
#pragma unroll
            for (int v = 0; v < VPT; ++v) h[v] = widen<T, VEC>(px[v]);
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) take(h[v], c0 + v * step);
    } else {
        for (int c = c0; c < A.D; c += step) take(sum_at(c), c);
    }
    const float2 sm = row_reduce<OUT == kRowCodes, false>(acc.sum(), m, buf);
    const float rstd = rsqrtf(sm.x * A.inv_D + A.eps);
    const float scale = fmaxf(sm.y * rstd * (1.f / kE4m3Max), kTinyScale), inv = __frcp_rn(scale);
    if (tid == 0) {
        if (A.rstd) A.rstd[row] = rstd;
        if (OUT == kRowCodes) A.scales[row] = scale;
    }
    if (VPT) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) finish_pack<T, VEC, OUT, HOW>(A, h[v], row, c0 + v * step, rstd, inv);
    } else {
        // whole steps, so that the lanes that share a scale stay together
        for (int c = c0; c - c0 < A.D + VEC; c += step) finish_pack<T, VEC, OUT, HOW>(A, sum_at(c), row, c, rstd, inv);
    }
}

__device__ __forceinline__ void copy_async(uint4* to, const void* from, uint32_t bytes)  // the rest of 16 bytes: zeros
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "r"(bytes) : "memory");
}

// Rows blockIdx.x blockDim.y + threadIdx.y, then a whole grid of rows further (a multiple of VEC of them, so that
// a thread's columns stay): a thread keeps its columns, their weights and their part of dweight in registers
// over all its rows.  Packs come through a ring of rows in shared memory, where every thread copies and
// reads places of its own, so that the rows in flight need neither registers nor barriers.
// RING = 0, for tensors off their 16 bytes: every pack is read directly.
// LEAN, for the longest rows: no more than dweight's part stays in registers; the weights are in shared memory,
// and the ring is read twice.
template <typename T, int VPT, int RING, int HOW>
__global__ void __maxnreg__(112) rms_backward_kernel(const RmsBwd A)
{
    constexpr int VEC = 16 / (int)sizeof(T), HELD = VPT * VEC > 16 ? 1 : VPT;
    static_assert(kNumSMs % VEC == 0, "a grid of kNumSMs CTAs is a multiple of VEC rows: a thread's columns stay");
    constexpr bool LEAN = VPT * VEC > 16;
    constexpr int kPart = HOW == kWhole ? kWhole : kSingle;  // a part's rows begin anywhere
    extern __shared__ uint4 ring[];  // [RING][3 VPT][threads], LEAN: weights [VPT][VEC / 4][threads]; at the end, as floats, [blockDim.y][D]
    __shared__ float2 buf[2][kRingThreads / 32];
    const int tid = threadIdx.x, step = blockDim.x * VEC;
    const int threads = blockDim.x * blockDim.y, own = threadIdx.y * blockDim.x + tid;
    begin_after();
    const long long all = (long long)gridDim.x * blockDim.y, row0 = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    const int lead = HOW != kWhole ? pack_lead(row0, A.D, VEC) : 0, c0 = tid * VEC - lead;
    const T *h = (const T*)A.h, *dy = (const T*)A.dy, *dh = (const T*)A.dh;
    auto fetch = [&](long long row, int slot) {
        if (row < A.rows) {
            uint4* to = ring + (size_t)slot * 3 * VPT * threads + own;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const PackCopy p = ring_copy(c0 + v * step, lead, A.D, VEC, (int)sizeof(T));
                copy_async(to + (3 * v) * threads, h + row * A.hs + p.at, p.bytes);
                copy_async(to + (3 * v + 1) * threads, dy + row * A.dys + p.at, p.bytes);
                if (dh) copy_async(to + (3 * v + 2) * threads, dh + row * A.D + p.at, p.bytes);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    constexpr bool vec = RING > 0;
    if constexpr (vec) {
#pragma unroll
        for (int i = 0; i < RING - 1; ++i) fetch(row0 + i * all, i);
    }
    float4* weights = reinterpret_cast<float4*>(ring + (vec ? (size_t)RING * 3 * VPT * threads : 0)) + own;
    auto weight = [&](int v) {
        Nums<VEC> r;
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 x = weights[(v * (VEC / 4) + i / 4) * threads];
            r.set(i, x.x, x.y);
            r.set(i + 2, x.z, x.w);
        }
        return r;
    };
    Nums<VEC> w[HELD], dw[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const Nums<VEC> wv = ld_weight<VEC, HOW>(A.w, A.w_dtype, c0 + v * step, A.D, A.w_vec);
        if (LEAN) {
#pragma unroll
            for (int i = 0; i < VEC; i += 4) {
                const float2 a = wv.pair(i), b = wv.pair(i + 2);
                weights[(v * (VEC / 4) + i / 4) * threads] = make_float4(a.x, a.y, b.x, b.y);
            }
        } else {
            w[LEAN ? 0 : v] = wv;
        }
        dw[v].fill(0.f);
    }
    int set = 0, slot = 0;
    float next_rstd = row0 < A.rows ? ld_plain(A.rstd + row0) : 0.f;
    for (long long row = row0; row < A.rows; row += all, set ^= 1, slot = vec ? (slot + 1) % (RING ? RING : 1) : 0) {
        const float rstd = next_rstd;
        if (row + all < A.rows) next_rstd = ld_plain(A.rstd + row + all);
        if constexpr (vec) {
            fetch(row + (RING - 1) * all, (slot + RING - 1) % RING);
            asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
        }
        const uint4* from = ring + (size_t)slot * 3 * VPT * threads + own;
        // pack v of h (0), dy (1) or dh (2); in the row's first pack, the neighbouring row's elements are zeros
        auto pack = [&](int v, int which) -> uint4 {
            const int c = c0 + v * step;
            if constexpr (!vec) {
                const T* src = which == 0 ? h + row * A.hs : which == 1 ? dy + row * A.dys : dh + row * A.D;
                return ld_cols<T, VEC, HOW>(src, c, A.D, false);
            }
            uint4 x = from[(3 * v + which) * threads];
            if (HOW != kWhole && c < 0) x = cut_pack<T>(x, -c, VEC);
            return x;
        };
        Nums<VEC> n[HELD], t[HELD], acc;
        uint4 pg[HELD];
        acc.fill(0.f);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int k = LEAN ? 0 : v;
            n[k] = mul(widen<T, VEC>(pack(v, 0)), rstd);
            t[k] = widen<T, VEC>(pack(v, 1));
            if (!LEAN && dh) pg[k] = pack(v, 2);
            dw[v] = fma(t[k], n[k], dw[v]);
            t[k] = mul(t[k], LEAN ? weight(v) : w[k]);
            acc = fma(t[k], n[k], acc);
        }
        const float c = -rstd * (row_reduce<false, true>(acc.sum(), 0.f, buf[set] + threadIdx.y * (blockDim.x >> 5)).x * A.inv_D);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int k = LEAN ? 0 : v;
            if (LEAN) {
                n[k] = mul(widen<T, VEC>(pack(v, 0)), rstd);
                t[k] = mul(widen<T, VEC>(pack(v, 1)), weight(v));
                if (dh) pg[k] = pack(v, 2);
            }
            Nums<VEC> o;
            if (dh) o = fma(t[k], rstd, widen<T, VEC>(pg[k]));
            else o = mul(t[k], rstd);
            st_cols<T, VEC, HOW>((T*)A.dx + row * A.D, c0 + v * step, A.D, fma(n[k], c, o));
        }
    }
    if (!A.part) return;
    float* out = A.part + (size_t)blockIdx.x * A.D;
    if (blockDim.y > 1) {
        float* sums = reinterpret_cast<float*>(ring);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();  // the ring is read
#pragma unroll
        for (int v = 0; v < VPT; ++v) st_cols<float, VEC, kPart>(sums + (size_t)threadIdx.y * A.D, c0 + v * step, A.D, dw[v]);
        __syncthreads();
        for (int c = own; c < A.D; c += threads) {
            float t = 0.f;
            for (int r = 0; r < (int)blockDim.y; ++r) t += sums[(size_t)r * A.D + c];
            out[c] = t;
        }
    } else {
#pragma unroll
        for (int v = 0; v < VPT; ++v) st_cols<float, VEC, kPart>(out, c0 + v * step, A.D, dw[v]);
    }
}

// Rows that registers do not hold: dx row by row, read twice; dweight's parts by the kernel below.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) rms_backward_long_kernel(const RmsBwd A)
{
    __shared__ float2 buf[32];
    const long long row = blockIdx.x;
    begin_after();
    const T *h = (const T*)A.h + row * A.hs, *dy = (const T*)A.dy + row * A.dys;
    const T* dh = A.dh ? (const T*)A.dh + row * A.D : nullptr;
    const float rstd = ld_plain(A.rstd + row);
    float s = 0.f;
    for (int c = threadIdx.x; c < A.D; c += blockDim.x)
        s = fmaf(to_f32(dy[c]) * (A.w ? ld_any(A.w, c, A.w_dtype) : 1.f), to_f32(h[c]) * rstd, s);
    const float m = row_reduce<false, false>(s, 0.f, buf).x * A.inv_D;
    for (int c = threadIdx.x; c < A.D; c += blockDim.x) {
        float o = rstd * fmaf(-(to_f32(h[c]) * rstd), m, to_f32(dy[c]) * (A.w ? ld_any(A.w, c, A.w_dtype) : 1.f));
        if (dh) o += to_f32(dh[c]);
        ((T*)A.dx)[row * A.D + c] = from_f32<T>(o);
    }
}

// CTAs (256 columns, a part of the rows): the columns along x, since a grid's y ends at 65535.
template <typename T>
__global__ void __launch_bounds__(256) rms_dweight_long_kernel(const RmsBwd A)
{
    const int c = blockIdx.x * 256 + threadIdx.x;
    begin_after();
    if (c >= A.D) return;
    float t = 0.f;
    for (long long row = blockIdx.y; row < A.rows; row += gridDim.y)
        t = fmaf(to_f32(((const T*)A.dy)[row * A.dys + c]), to_f32(((const T*)A.h)[row * A.hs + c]) * ld_plain(A.rstd + row), t);
    A.part[(size_t)blockIdx.y * A.D + c] = t;
}

// dweight = the parts' sum, 8 columns a CTA, 16 threads over the parts of each.  Small CTAs: they are
// resident beside the rows' CTAs (which leave them an eighth of the registers) before those end.
__global__ void __launch_bounds__(128) rms_dweight_sum_kernel(const float* part, int parts, int D, float* dweight)
{
    __shared__ float s[16][9];
    const int col = threadIdx.x & 7, g = threadIdx.x >> 3, c = blockIdx.x * 8 + col;
    tc::grid_dep_wait();
    float t = 0.f;
    if (c < D) {
#pragma unroll 10
        for (int p = g; p < parts; p += 16) t += __ldcg(part + (size_t)p * D + c);
    }
    s[g][col] = t;
    __syncthreads();
    if (threadIdx.x < 8 && c < D) {
        t = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += s[i][threadIdx.x];
        dweight[c] = t;
    }
}

// How a row is laid over threads: tpr threads of vpt packs (0: more than registers hold), ry rows a CTA.  It, and with
// it the order of every sum, goes by D, the rows and the types alone: the same numbers give the same bits
// whatever their alignment and strides (packs off their 16 bytes are loaded one by one).
struct Shape {
    int vpt, tpr, ry;
};

// `most`: packs of a thread; a thread takes one more while the row has more than `threads` times as many.
Shape shape_of(const rms_params_t* p, int most, int threads, int max_threads)
{
    const int vec = 16 / (int)elem_size(p->x_dtype);
    const int64_t packs = (p->D + (p->D % vec ? vec - 1 : 0) + vec - 1) / vec;
    Shape s{1, 0, 1};
    while (s.vpt < most && packs > threads * (int64_t)s.vpt) ++s.vpt;
    const int64_t t = ((packs + s.vpt - 1) / s.vpt + 31) / 32 * 32;
    if (t > max_threads) s.vpt = 0;
    s.tpr = t > max_threads ? max_threads : (int)t;
    return s;
}

// Forward: a CTA a row, 256 threads before a thread takes a second pack; short rows (up to 16 elements a
// lane) a warp each, several to a CTA where there are many.
Shape fwd_shape(const rms_params_t* p)
{
    const bool shorter = p->D <= 512;
    Shape s = shape_of(p, 4, shorter ? 32 : 256, kMaxThreads);
    if (s.tpr == 32) {
        s.ry = 8;
        while (s.ry > 1 && p->rows < (int64_t)s.ry * 2 * kNumSMs) s.ry /= 2;
    }
    return s;
}

// Backward: a row's exchange between threads costs as much as 16 elements' arithmetic, so 16 elements a
// thread, for longer rows three packs of 16-bit elements; one CTA of up to 512 threads an SM.
Shape bwd_shape(const rms_params_t* p)
{
    const int most = p->x_dtype == GDN_F32 ? 4 : 2;
    Shape s = shape_of(p, most, 32, kRingThreads);
    if (s.vpt == 0 && most < 3) s = shape_of(p, 3, 32, kRingThreads);
    if (s.vpt > 0) {
        s.ry = kRingThreads / s.tpr;
        while (s.ry > 1 && p->rows < (int64_t)s.ry * kNumSMs) s.ry /= 2;
    }
    return s;
}

template <typename T, int VPT>
int launch_fwd_v(const RmsFwd& A, const Shape& s, cudaStream_t st)
{
    const unsigned grid = (unsigned)((A.rows + s.ry - 1) / s.ry);
    const dim3 block(s.tpr, s.ry);
    // a cut pack may reach into the next row, but not past it: rows shorter than a pack are read element by element
    constexpr int VEC = 16 / (int)sizeof(T);
    const int how = !A.vec || A.D < VEC ? kSingle : A.D % VEC != 0 ? kCut : kWhole;
    void (*kernel)(RmsFwd);
    if (A.y_dtype != RMS_E4M3)
        kernel = how == kWhole ? rms_forward_kernel<T, VPT, kPlain, kWhole> : how == kCut ? rms_forward_kernel<T, VPT, kPlain, kCut> : rms_forward_kernel<T, VPT, kPlain, kSingle>;
    else if (!A.lg_group)
        kernel = how == kWhole ? rms_forward_kernel<T, VPT, kRowCodes, kWhole> : how == kCut ? rms_forward_kernel<T, VPT, kRowCodes, kCut> : rms_forward_kernel<T, VPT, kRowCodes, kSingle>;
    else  // groups of columns divide D into whole packs
        kernel = how == kWhole ? rms_forward_kernel<T, VPT, kGroupCodes, kWhole> : rms_forward_kernel<T, VPT, kGroupCodes, kSingle>;
    return launch_after(kernel, grid, block, 0, st, A);
}

template <typename T>
int launch_fwd(const RmsFwd& A, const Shape& s, cudaStream_t st)
{
    switch (s.vpt) {
        case 1: return launch_fwd_v<T, 1>(A, s, st);
        case 2: return launch_fwd_v<T, 2>(A, s, st);
        case 3: return launch_fwd_v<T, 3>(A, s, st);
        case 4: return launch_fwd_v<T, 4>(A, s, st);
        default: return launch_fwd_v<T, 0>(A, s, st);
    }
}

template <typename T, int VPT>
int launch_bwd_v(const RmsBwd& A, const Shape& s, int ctas, cudaStream_t st)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    const size_t row = (size_t)3 * VPT * s.tpr * s.ry * 16;  // of a ring: 96 KB at most
    const size_t weights = VPT * VEC > 16 ? (size_t)VPT * VEC * 4 * s.tpr * s.ry : 0;
    const bool deep = 4 * row + weights <= 200 * 1024, cut = A.D % VEC != 0;
    size_t smem = weights + (A.vec ? (deep ? 4 : 2) * row : 0);
    if (A.part && s.ry > 1 && smem < (size_t)s.ry * A.D * 4) smem = (size_t)s.ry * A.D * 4;
    if (smem > kMostSmem) return (int)cudaErrorInvalidValue;  // not for the shapes of bwd_shape()
    const auto kernel = !A.vec ? rms_backward_kernel<T, VPT, 0, kSingle>
                        : deep ? (cut ? rms_backward_kernel<T, VPT, 4, kCut> : rms_backward_kernel<T, VPT, 4, kWhole>)
                               : (cut ? rms_backward_kernel<T, VPT, 2, kCut> : rms_backward_kernel<T, VPT, 2, kWhole>);
    // the limit is the kernel's, not the call's: every call sets the same, so that none lowers another thread's
    if (smem > 40 * 1024) {
        const int e = (int)cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (e) return e;
    }
    return launch_after(kernel, ctas, dim3(s.tpr, s.ry), smem, st, A);
}

template <typename T>
int launch_bwd(const RmsBwd& A, const Shape& s, int ctas, cudaStream_t st)
{
    switch (s.vpt) {
        case 1: return launch_bwd_v<T, 1>(A, s, ctas, st);
        case 2: return launch_bwd_v<T, 2>(A, s, ctas, st);
        case 3: return launch_bwd_v<T, 3>(A, s, ctas, st);
        case 4: if constexpr (sizeof(T) == 4) return launch_bwd_v<T, 4>(A, s, ctas, st);
    }
    const int e = launch_after(rms_backward_long_kernel<T>, (unsigned)A.rows, kMaxThreads, 0, st, A);
    if (e || !A.part) return e;
    return launch_after(rms_dweight_long_kernel<T>, dim3((A.D + 255) / 256, ctas), 256, 0, st, A);
}

// CTAs of the backward, each with its own part of dweight.
int bwd_ctas(const rms_params_t* p, const Shape& s)
{
    const int64_t need = (p->rows + s.ry - 1) / s.ry;
    return (int)(need < kNumSMs ? need : kNumSMs);
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

// Packs of 16 bytes are aligned in every tensor that has rows.
bool packs_ok(const rms_params_t* p, std::initializer_list<const void*> ptrs)
{
    const int vec = 16 / (int)elem_size(p->x_dtype);
    for (const void* q : ptrs)
        if ((uintptr_t)q % 16 != 0) return false;
    return (p->x_s - p->D) % vec == 0 && (p->res_s - p->D) % vec == 0;
}
}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" size_t rms_backward_workspace_bytes(const rms_params_t* p)
{
    if (check(p) != GDN_OK || p->rows == 0) return 0;
    return (size_t)bwd_ctas(p, bwd_shape(p)) * p->D * 4;
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
    A.w_dtype = p->w_dtype; A.y_dtype = p->y_dtype; A.lg_group = e4 && p->group ? (p->group == 16 ? 4 : p->group == 32 ? 5 : p->group == 64 ? 6 : 7) : 0;
    A.eps = p->eps; A.inv_D = 1.f / (float)p->D;
    A.vec = packs_ok(p, {x, residual, h, y});
    A.w_vec = (uintptr_t)weight % 16 == 0;
    const Shape s = fwd_shape(p);
    cudaStream_t cs = (cudaStream_t)stream;
    int e;
    if (p->x_dtype == GDN_F32) e = launch_fwd<float>(A, s, cs);
    else if (p->x_dtype == GDN_BF16) e = launch_fwd<__nv_bfloat16>(A, s, cs);
    else e = launch_fwd<__half>(A, s, cs);
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
    A.vec = packs_ok(p, {h, dy, dh, dx});
    A.w_vec = (uintptr_t)weight % 16 == 0;
    const Shape s = bwd_shape(p);
    const int ctas = bwd_ctas(p, s);
    int e;
    if (p->x_dtype == GDN_F32) e = launch_bwd<float>(A, s, ctas, cs);
    else if (p->x_dtype == GDN_BF16) e = launch_bwd<__nv_bfloat16>(A, s, ctas, cs);
    else e = launch_bwd<__half>(A, s, ctas, cs);
    if (!e && dweight) {
        e = launch_after(rms_dweight_sum_kernel, (unsigned)((p->D + 7) / 8), 128, 0, cs, (const float*)A.part, ctas, A.D, dweight);
    }
    return e ? cuda_fail(e, "rms_backward launch") : GDN_OK;
}
