"""The index arithmetic that kernels and host share (csrc/gdn_packs.h), compiled for the host: every address that a
kernel forms from it, for every thread, lies on 16 bytes and inside its tensor."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HARNESS = r"""
#include "gdn_packs.h"
using namespace gdn;

// The copies of one row by `threads` threads of `vpt` packs: 0 where all is well, else 1 + the kind of mistake.
// Rows lie `stride` elements apart; total: the tensor's elements.
extern "C" int norm_ring_row(long long row, int D, long long stride, long long total, int vec, int elem_bytes, int threads, int vpt)
{
    const int lead = pack_lead(row, D, vec);
    const long long first = row * stride;
    long long next = -lead;  // the packs that have bytes follow each other and cover the row
    for (int v = 0; v < vpt; ++v)
        for (int t = 0; t < threads; ++t) {
            const int c = (v * threads + t) * vec - lead;
            const PackCopy p = ring_copy(c, lead, D, vec, elem_bytes);
            if ((first + p.at) * elem_bytes % 16 != 0) return 1;            // asynchronous copies start on 16 bytes
            if (first + p.at < 0 || first + p.at >= total) return 2;
            if (p.bytes > 16 || first + p.at + (long long)p.bytes / elem_bytes > total) return 3;
            if (c < D && (p.at != next || p.at + (int)p.bytes / elem_bytes > D)) return 4;
            if (c < D) next = c + vec;
            if (c >= D && p.bytes != 0) return 5;
        }
    return next >= D ? 0 : 6;
}

// A row of V elements, the first `lead` past a 16-byte boundary, in `splits` segments of `seg`: 0 where the
// segments' elements follow each other and are the row's, else 1 + the kind of mistake.  Long rows: the first and
// last segments.
extern "C" int selection_row(int V, int lead, int splits, int seg, int vec)
{
    for (long long s = 0; s < splits; s = s == 40 && splits > 200 ? splits - 40 : s + 1) {
        const PackSegment p = pack_segment((unsigned)s, seg, (unsigned)lead, V);
        long long lo = s * seg - lead, end = lo + seg;  // columns, in more than 32 bits
        if (lo < 0) lo = 0;
        if (end > V) end = V;
        if (end < lo) end = lo;
        const long long first = (long long)p.first - lead;
        if (p.first != (unsigned long long)s * seg || p.end < 0 || p.end > seg || p.lo < 0 || p.lo >= vec) return 1;
        if (lo < end && (first + p.lo != lo || first + p.end != end)) return 2;
        if (lo == end && p.end > p.lo) return 3;
        // the column of an element in the kernel's 32-bit arithmetic
        if (lo < end && (p.first - (unsigned)lead) + (unsigned)(p.end - 1) != (unsigned long long)(end - 1)) return 4;
    }
    return (long long)splits * seg - lead >= V ? 0 : 5;
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("packs")
    (d / "packs.cpp").write_text(HARNESS)
    lib = str(d / "libpacks.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "gated_delta_rule_backward_gb300", "csrc"), str(d / "packs.cpp"), "-o", lib], check=True)
    return ctypes.CDLL(lib)


@pytest.mark.parametrize("elem_bytes", [2, 4])
def test_norm_ring_copies_are_aligned_and_inside(host, elem_bytes):
    """Rows of every length class over the threads that the gradient gives them (multiples of 32, with packs to spare)."""
    vec, i64 = 16 // elem_bytes, ctypes.c_longlong
    for D in [1, 2, 3, 7, 8, 9, 31, 96, 100, 127, 1000, 1001, 2047, 2048, 4090, 4095, 4096, 8189, 8191, 12285, 12288]:
        packs = (D + vec - 1 + vec - 1) // vec
        for vpt in (1, 2, 3, 4):
            threads = ((packs + vpt - 1) // vpt + 31) // 32 * 32
            for rows, stride in ((40, D), (40, D + 5 * vec)):
                total = (rows - 1) * stride + D
                for row in list(range(17)) + [rows - 1]:
                    got = host.norm_ring_row(i64(row), D, i64(stride), i64(total), vec, elem_bytes, threads, vpt)
                    assert got == 0, (D, vpt, rows, stride, row, got)


@pytest.mark.parametrize("vec", [4, 8])
def test_selection_segments_cover_a_row_of_any_length(host, vec):
    for V in [1, 2, 7, 8, 9, 63, 1000, 4096, 32000, 50001, 128257, 2**24 + 1, 2**30, 2**31 - 20000, 2**31 - 9, 2**31 - 8, 2**31 - 2, 2**31 - 1]:
        for lg_packs in (1, 2, 3):   # as the plan of a selection cuts rows: segments of one size, whole packs
            span, most = V + vec - 1, (vec * 256) << lg_packs
            splits = -(-span // most)
            seg = -(-span // (splits * vec)) * vec
            for lead in range(vec):
                got = host.selection_row(V, lead, splits, seg, vec)
                assert got == 0, (V, lg_packs, lead, got)
