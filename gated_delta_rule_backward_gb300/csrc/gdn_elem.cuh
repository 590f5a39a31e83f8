// gdn_elem.cuh -- storage types (fp32, bf16, fp16): loads that widen exactly to fp32 and stores
// that round once to nearest even, for the kernels that take 16-bit tensors as they are.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/gdn.h"
#include "gdn_f32x2.cuh"

namespace gdn {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// The hardware's 2^x (2^-22 relative; 0 below 2^-126).
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two neighbours, widened together.
__device__ __forceinline__ f2 widen2(const float* p) { return pack2(p[0], p[1]); }
__device__ __forceinline__ f2 widen2(const __nv_bfloat16* p)
{
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ f2 widen2(const __half* p)
{
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(p));
    return pack2(v.x, v.y);
}

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// A plain load.  A load through the path for constant data (`ld.global.nc`) would be a promise that nobody writes
// there while this kernel runs, which launch_after() does not keep: the kernel starts beside the one that may still be
// writing it, and the compiler may lift such a load above the wait.
template <typename V>
__device__ __forceinline__ V ld_plain(const V* p) { return *p; }

// One element of a tensor whose type is only known at run time (gdn_dtype_t).
__device__ __forceinline__ float ld_any(const void* p, long long i, int dtype)
{
    if (dtype == GDN_F32) return ld_plain((const float*)p + i);
    if (dtype == GDN_BF16) return __bfloat162float(ld_plain((const __nv_bfloat16*)p + i));
    return __half2float(ld_plain((const __half*)p + i));
}
__device__ __forceinline__ void st_any(void* p, long long i, int dtype, float x)
{
    if (dtype == GDN_F32) ((float*)p)[i] = x;
    else if (dtype == GDN_BF16) ((__nv_bfloat16*)p)[i] = __float2bfloat16_rn(x);
    else ((__half*)p)[i] = __float2half_rn(x);
}

// VEC consecutive elements as one load where `vec` says that they are aligned for it; kept as they are
// stored until get() widens them, so that a load in flight holds few registers.
template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Pack {
    T x[VEC];
    __device__ __forceinline__ float get(int i) const { return to_f32(x[i]); }
    // Elements i and i + 1 (i even) for the packed fp32 instructions.
    __device__ __forceinline__ f2 pair(int i) const { return widen2(x + i); }
};

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> ld_pack(const T* p, bool vec)
{
    Pack<T, VEC> r;
    constexpr int B = (int)sizeof(T) * VEC;
    static_assert(B == 4 || B == 8 || B == 16, "one load of 4, 8 or 16 bytes");
    if (vec) {
        if (B == 16) *reinterpret_cast<uint4*>(&r) = ld_plain(reinterpret_cast<const uint4*>(p));
        else if (B == 8) *reinterpret_cast<uint2*>(&r) = ld_plain(reinterpret_cast<const uint2*>(p));
        else *reinterpret_cast<uint32_t*>(&r) = ld_plain(reinterpret_cast<const uint32_t*>(p));
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.x[i] = ld_plain(p + i);
    }
    return r;
}

inline size_t elem_size(int dtype) { return dtype == GDN_F32 ? 4 : 2; }
inline bool known_dtype(int dtype) { return dtype == GDN_F32 || dtype == GDN_BF16 || dtype == GDN_F16; }

}  // namespace gdn
