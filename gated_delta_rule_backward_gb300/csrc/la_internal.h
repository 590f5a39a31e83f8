// la_internal.h -- linear attention's one core, which the forward pass and each of the backward pass's products are
// runs of (include/la.h; not part of the C ABI).
//
// Forwards in time:   S_t = a_t S_{t-1} + cs z_t y_t^T,      out_t = co S_t x_t          (S: DV x DK)
// backwards:          S_t = a_{t+1} S_{t+1} + cs z_t y_t^T,  out_t = co S_t x_t,         and after token 0 S <- a_0 S
//     y:  (x, y, z) = (q, k, v)   forwards,  co = scale
//     dq: (dy, v, k)              forwards,  co = scale, S the transposed state
//     dk: (v, dy, q)              backwards, cs = scale, S the transposed gradient
//     dv: (k, q, dy)              backwards, cs = scale
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/la.h"

namespace gdn {

struct LaRun {
    const void *x, *y, *z, *g;
    long long xs0, xs1, ys0, ys1, zs0, zs1, gs0, gs1;  // element strides of {token, head}
    int xh, yh, zh;                                    // heads of each: value head h takes h mod these
    int gate_dtype, out_dtype;
    const int* cu;  // may be null
    int T, n_tok, n_seq, H, DK, DV;
    const float* s_in;    // null: zeros
    const int* slot_in;   // null: state n is sequence n's
    float* s_out;         // null: nowhere
    const int* slot_out;  // null as above
    long long in_stride, out_stride;  // elements between states (of H heads)
    int n_slots;
    int transposed_in, transposed_out;  // a state's element (row j, column i) lies at i DV + j, not j DK + i
    int reverse;
    float co, cs;
    void* out;  // [n_tok][H][DV]
    // Token form: 0, or segments of `per` tokens of each sequence's walk that start from what those before left (transposed, the
    // first's with the state before it) and their decays; states[.][0] is the state before the first.
    int segments, per;
    const float *states, *decays;  // [n_seq H][segments][DK][DV], [n_seq H][segments]
    int held;  // self-test of the chunked form: 1 for a hand-over, the gates', that waits for an arrival too many
};

// The token rows of sequence n, and the states that it starts from and leaves (-1: none).
struct LaSequence {
    long long lo, hi;
    int in, out;
    bool ok;
};

constexpr float kLaLeastGate = -104.f;  // exp of it is 0 in fp32
constexpr float kLaMostGate = 1000.f;    // exp of it is infinite

#if defined(__CUDACC__)
__device__ __forceinline__ LaSequence la_sequence(const LaRun& A, int n)
{
    LaSequence s;
    s.in = A.slot_in ? A.slot_in[n] : n;
    s.out = A.slot_out ? A.slot_out[n] : n;
    s.lo = A.cu ? A.cu[n] : (long long)n * A.T;
    s.hi = A.cu ? A.cu[n + 1] : s.lo + A.T;
    s.ok = s.lo >= 0 && s.hi >= s.lo && s.hi <= A.n_tok && s.hi - s.lo <= A.T && (!A.slot_in || (s.in >= -1 && s.in < A.n_slots)) &&
           (!A.slot_out || (s.out >= -1 && s.out < A.n_slots));
    if (!A.s_in) s.in = -1;
    if (!A.s_out) s.out = -1;
    return s;
}
#endif

// Launchers: a cudaError_t as int.  dtype: of x, y and z.
int launch_la_token(const LaRun& A, int dtype, cudaStream_t stream);

// The chunked form (la_chunk.cu).
bool la_chunk_fits(const la_params_t* p);
size_t la_chunk_workspace(const LaRun& A);  // bytes
size_t la_tokens_workspace(const LaRun& A);
int launch_la_tokens(const LaRun& run, int dtype, void* workspace, cudaStream_t st);  // the token form by segments, of the chunked form's sizes
int launch_la_chunk(const LaRun& A, void* workspace, cudaStream_t stream);

// n status words in one copy, and one of them set to 0.
int la_read_words(const void* symbol, void* stream, int n, int* words);
int la_clear_word(const void* symbol, void* stream, int i);
// Read and clear: waits that gave up, and, where there were none and bad_too, bad slots and token ranges.
int la_chunk_take_status(void* stream, bool bad_too, int* timeout, int* bad);
int la_token_take_status(void* stream, int* bad);

}  // namespace gdn
