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

// Segment `split` of `seg` elements (whole packs) of a row of V whose first element is `lead` past a 16-byte boundary:
// the segment begins `first` elements after that boundary, and of its elements those from lo to below end are the
// row's.  Unsigned, since what the last segments reach to passes 2^31 for the longest rows.
struct PackSegment {
    unsigned first;
    int lo, end;
};
GDN_PACKS_FN PackSegment pack_segment(unsigned split, int seg, unsigned lead, int V)
{
    const unsigned first = split * (unsigned)seg, all = (unsigned)V + lead, left = first < all ? all - first : 0u;
    return {first, split == 0 ? (int)lead : 0, left < (unsigned)seg ? (int)left : seg};
}

}  // namespace gdn
