// gdn_packs.h -- index arithmetic of rows that are read in packs of 16 bytes, for the kernels and, since nothing in it
// needs a GPU, for the host.
#pragma once

#if defined(__CUDACC__)
#define GDN_PACKS_FN __host__ __device__ __forceinline__
#else
#define GDN_PACKS_FN inline
#endif

namespace gdn {

// Packs at multiples of `vec` elements of the flat index row D + column: where row `row` begins in its first pack.
// vec: a power of two.
GDN_PACKS_FN int pack_lead(long long row, int D, int vec) { return (int)(((unsigned)row * (unsigned)D) & (unsigned)(vec - 1)); }

// The asynchronous copy of the pack at column c of a row of D into a ring: where it reads from (an element of the row,
// from -lead on, which lies on 16 bytes as c does) and how many bytes (the rest of the 16 are zeros).  A pack past the
// row's end is a copy of no bytes, whose address has to be aligned all the same: the row's first pack's.
struct PackCopy {
    int at;
    unsigned bytes;
};
GDN_PACKS_FN PackCopy ring_copy(int c, int lead, int D, int vec, int elem_bytes)
{
    if (c >= D) return {-lead, 0u};
    return {c, c + vec <= D ? 16u : (unsigned)((D - c) * elem_bytes)};
}

}  // namespace gdn
