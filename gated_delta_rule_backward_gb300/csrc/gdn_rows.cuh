// gdn_rows.cuh -- rows of logits read in packs of 16 bytes from any alignment, and what a softmax over them needs.
#pragma once

#include "gdn_elem.cuh"
#include "gdn_f32x2.cuh"
#include "gdn_packs.h"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

// exp(a - b) for a <= b, 1 where both are the same infinity.
__device__ __forceinline__ float exp_diff(float a, float b) { return a == b ? 1.f : ex2((a - b) * kLog2e); }

// The largest of a pack's elements; one that is NaN does not count.
__device__ __forceinline__ float pack_max(const Pack<float, 4>& v)
{
    return fmaxf(fmaxf(v.x[0], v.x[1]), fmaxf(v.x[2], v.x[3]));
}
__device__ __forceinline__ float pack_max(const Pack<__nv_bfloat16, 8>& v)
{
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(v.x);
    const float2 m = __bfloat1622float2(__hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3])));
    return fmaxf(m.x, m.y);
}
__device__ __forceinline__ float pack_max(const Pack<__half, 8>& v)
{
    const __half2* w = reinterpret_cast<const __half2*>(v.x);
    const float2 m = __half22float2(__hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3])));
    return fmaxf(m.x, m.y);
}

// A row's packs lie on 16-byte boundaries: it starts `lead` elements into the first.  Segment `split`
// begins at element split seg - lead; what is outside the row or the segment reads as -inf.
template <typename T>
struct Segment {
    const T* at;  // on 16 bytes
    unsigned column;  // of its first element, in unsigned arithmetic (the first segment may begin before the row)
    int lo, end;
};
template <typename T>
__device__ __forceinline__ Segment<T> segment_of(const T* row, int split, int seg, int V)
{
    const unsigned lead = (unsigned)(((uintptr_t)row & 15) / sizeof(T));
    const PackSegment s = pack_segment((unsigned)split, seg, lead, V);
    return {row - lead + s.first, s.first - lead, s.lo, s.end};
}
// N packs whose first elements are in(p) into a segment: the whole ones all in flight at once, then the elements of a
// pack that the row's first or last 16 bytes cut (in a loop of its own, so that the code that always runs stays short).
template <typename T, int VEC, int N, typename In>
__device__ __forceinline__ void ld_chunk_packs(Pack<T, VEC> (&x)[N], const Segment<T>& s, const In& in)
{
    Pack<T, VEC> none;
#pragma unroll
    for (int i = 0; i < VEC; ++i) none.x[i] = from_f32<T>(-INFINITY);
    unsigned cut = 0;
#pragma unroll
    for (int p = 0; p < N; ++p) {
        const int at = in(p);
        const bool inside = at < s.end, whole = at >= s.lo && at + VEC <= s.end;
        x[p] = none;
        if (whole) x[p] = ld_pack<T, VEC>(s.at + at, true);
        cut |= (inside && !whole ? 1u : 0u) << p;
    }
    while (cut) {
        const int c = __ffs(cut) - 1, at = in(c);
        cut &= cut - 1;
        Pack<T, VEC> part = none;
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (at + i >= s.lo && at + i < s.end) part.x[i] = s.at[at + i];
#pragma unroll
        for (int p = 0; p < N; ++p)
            if (p == c) x[p] = part;
    }
}

}  // namespace gdn
