// beam.cu -- a beam search's selection over beams and vocabulary (include/beam.h).
//
// Two kernels.  The first cuts every beam's row into segments, one a CTA, each read once into
// registers: the segment's maximum, the sum of exponentials against it, and its n best logits
// (the order within a row does not need the row's normaliser).  The second, one CTA a
// sequence, joins the segments' sums into each row's log-sum-exp, turns the K x segments x n
// kept logits into scores and selects among them.
//
// Selecting n of a CTA's items: the n-th largest of the threads' maxima is a bound that at
// least n items reach, and for items in no particular order few more do.  So: every warp
// gives its R largest thread maxima, the n-th largest of all of those is the bound, and the
// items that reach it go to a list (in any order).  A list that is still long goes through the same once
// more, now spread evenly over the threads.  Each listed item's rank is the number of
// listed keys above its own; keys are (value, lowest index first) in one 64-bit number, so ranks do not
// depend on the list's order.  Where more items reach the bound than the list holds (many
// equal values), n rounds of a block-wide maximum select instead.
#include <climits>
#include <cstdio>

#include "../../include/beam.h"
#include "gdn_elem.cuh"
#include "gdn_f32x2.cuh"
#include "gdn_internal.h"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxOut = 64, kMaxBeams = 64;
constexpr int kList = 1024, kLong = 96;  // items a list holds; items from which a second bound pays
constexpr int kItems = 16;               // keys that a thread of the join holds
constexpr unsigned kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

typedef unsigned long long u64;

struct BeamArgs {
    const void* logits;
    const float* scores;
    const uint8_t* done;
    const int* slots;
    float* scores_out;
    int *parent, *token, *src_slots;
    float2* sums;  // [N K][splits] maximum and sum of a segment
    u64* best;     // [N K][splits][n_out] its best (order(logit), ~index) keys, 0 past their number
    long long row_stride;
    int K, V, splits, seg, n, pad;
};

// Floats as whole numbers of the same order; -0 and +0 have to be the same float before.
__device__ __forceinline__ unsigned order(float x)
{
    const unsigned b = __float_as_uint(x);
    return b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unorder(unsigned o)
{
    return __uint_as_float(o ^ ((unsigned)((int)~o >> 31) | 0x80000000u));
}
constexpr unsigned kNegInf = 0x007fffffu;  // order(-inf)

__device__ __forceinline__ u64 key_of(unsigned o, unsigned index) { return (u64)o << 32 | (0xffffffffu - index); }

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// exp(a - b) for a <= b, 1 where both are the same infinity.
__device__ __forceinline__ float exp_diff(float a, float b) { return a == b ? 1.f : ex2((a - b) * kLog2e); }

struct SelectSmem {
    u64 list[2][kList];
    u64 warp_best[kWarps];
    u64 out[kMaxOut];
    __align__(16) unsigned top[kWarps * 8];
    int count[2];
};

// R: thread maxima that a warp gives for a selection of n.
__device__ __forceinline__ int tops_of(int n) { return n <= 16 ? 4 : 8; }

// A warp's R largest of its lanes' v (0: none), from high to low; returns the first.
__device__ __forceinline__ unsigned warp_tops(unsigned v, int R, unsigned* out, int lane)
{
    unsigned first = 0;
    for (int r = 0; r < R; ++r) {
        const unsigned best = __reduce_max_sync(kAll, v);
        if (r == 0) first = best;
        if (lane == 0) out[r] = best;
        const unsigned who = __ballot_sync(kAll, v == best);
        if (lane == __ffs(who) - 1) v = 0;
    }
    return first;
}

// The largest of the tops that n of them reach (0 when there is none): every warp finds it by itself.
__device__ __forceinline__ unsigned nth_top(const unsigned* top, int n, int lane)
{
    const uint4* all = reinterpret_cast<const uint4*>(top);
    unsigned best = 0;
    if (tops_of(n) == 4) {
        const unsigned v = top[lane];
        int reach = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const uint4 t = all[i];
            reach += (t.x >= v) + (t.y >= v) + (t.z >= v) + (t.w >= v);
        }
        best = reach >= n ? v : 0;
    } else {
        const unsigned v = top[lane], w = top[32 + lane];
        int rv = 0, rw = 0;
#pragma unroll
        for (int i = 0; i < 2 * kWarps; ++i) {
            const uint4 t = all[i];
            rv += (t.x >= v) + (t.y >= v) + (t.z >= v) + (t.w >= v);
            rw += (t.x >= w) + (t.y >= w) + (t.z >= w) + (t.w >= w);
        }
        best = max(rv >= n ? v : 0, rw >= n ? w : 0);
    }
    best = __reduce_max_sync(kAll, best);
    return best > kNegInf ? best : kNegInf + 1;  // an item at -inf is none
}

// The n best keys of the CTA's items into S.out (0 past their number), from high to low.  `each(bound, take)`
// calls take(order(value), index) for every item of this thread whose order reaches bound; `mine` is the largest.
// S.top holds the warps' tops and S.count 0, a barrier ago.  Ends with a barrier.
template <typename Each>
__device__ __forceinline__ void select_n(SelectSmem& S, int n, unsigned mine, const Each& each)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned bound = nth_top(S.top, n, lane);
    if (mine >= bound)
        each(bound, [&](unsigned o, unsigned index) {
            const int at = atomicAdd(&S.count[0], 1);
            if (at < kList) S.list[0][at] = key_of(o, index);
        });
    __syncthreads();
    int listed = S.count[0];
    if (listed <= kList) {
        const u64* list = S.list[0];
        if (listed > kLong) {
            unsigned best = 0;
            for (int t = tid; t < listed; t += kThreads) best = max(best, (unsigned)(S.list[0][t] >> 32));
            const int R = tops_of(n);
            warp_tops(best, R, S.top + warp * R, lane);
            __syncthreads();
            const unsigned closer = nth_top(S.top, n, lane);
            for (int t = tid; t < listed; t += kThreads) {
                const u64 key = S.list[0][t];
                if ((unsigned)(key >> 32) >= closer) S.list[1][atomicAdd(&S.count[1], 1)] = key;
            }
            __syncthreads();
            listed = S.count[1];
            list = S.list[1];
        }
        for (int t = tid; t < listed; t += kThreads) {
            const u64 key = list[t];
            int rank = 0;
            for (int i = 0; i < listed; ++i) rank += list[i] > key;
            if (rank < n) S.out[rank] = key;
        }
        for (int i = listed + tid; i < n; i += kThreads) S.out[i] = 0;
        __syncthreads();
        return;
    }
    u64 last = ~0ull;
    for (int r = 0; r < n; ++r) {
        u64 best = 0;
        if (mine >= bound)
            each(bound, [&](unsigned o, unsigned index) {
                const u64 key = key_of(o, index);
                if (key < last && key > best) best = key;
            });
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            const u64 other = __shfl_xor_sync(kAll, best, o);
            best = other > best ? other : best;
        }
        if (lane == 0) S.warp_best[warp] = best;
        __syncthreads();
        last = 0;
        for (int i = 0; i < kWarps; ++i) last = S.warp_best[i] > last ? S.warp_best[i] : last;
        if (tid == 0) S.out[r] = last;
        __syncthreads();
    }
}

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

// PACKS loads of 16 bytes a thread.
template <typename T, int PACKS>
__global__ void __launch_bounds__(kThreads, PACKS == 8 ? 3 : 4) beam_segment_kernel(const BeamArgs A)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    __shared__ SelectSmem S;
    __shared__ float2 part[kWarps];
    const int row = blockIdx.x / A.splits, split = blockIdx.x - row * A.splits;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    tc::grid_dep_launch();
    if ((A.done && A.done[row]) || !(A.scores[row] > -INFINITY)) return;

    // The segment's packs lie on 16-byte boundaries: the row starts `lead` elements into the first.
    const T* base = (const T*)A.logits + row * A.row_stride;
    const int lead = (int)(((uintptr_t)base & 15) / sizeof(T));
    const int first = split * A.seg - lead;
    Pack<T, VEC> x[PACKS];
#pragma unroll
    for (int p = 0; p < PACKS; ++p) {
        const int in = (p * kThreads + tid) * VEC, at = first + in;
        if (in < A.seg && at >= 0 && at + VEC <= A.V) {
            x[p] = ld_pack<T, VEC>(base + at, true);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[p].x[i] = in < A.seg && at + i >= 0 && at + i < A.V ? base[at + i] : from_f32<T>(-INFINITY);
        }
    }
    float top[PACKS], m = -INFINITY;
#pragma unroll
    for (int p = 0; p < PACKS; ++p) {
        top[p] = fmaxf(pack_max(x[p]), -INFINITY);  // a pack of NaNs
        m = fmaxf(m, top[p]);
    }
    // The sum against the thread's own maximum: (x - m) log2 e in two roundings, then the exponential.
    float s = 0.f;
    if (m < INFINITY && m > -INFINITY) {
        f2 s2 = 0;
        const f2 mm = pack2(-m, -m), ll = pack2(kLog2e, kLog2e);
#pragma unroll
        for (int p = 0; p < PACKS; ++p)
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                const float2 v = unpack2(mul2(add2(pack2(x[p].get(i), x[p].get(i + 1)), mm), ll));
                s2 = add2(s2, pack2(ex2(v.x), ex2(v.y)));
            }
        s = sum2(s2);
    }
    if (m == INFINITY || s != s) {  // infinities share the probability; NaNs are left out
        s = 0.f;
#pragma unroll
        for (int p = 0; p < PACKS; ++p)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float v = x[p].get(i);
                s += v == m ? 1.f : v < m ? ex2((v - m) * kLog2e) : 0.f;
            }
    }
    const unsigned mine = order(m + 0.f);  // + 0: -0 becomes 0
    const int R = tops_of(A.n);
    if (tid < 2) S.count[tid] = 0;
    const float wm = unorder(warp_tops(mine, R, S.top + warp * R, lane));
    s = m > -INFINITY ? s * exp_diff(m, wm) : 0.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    if (lane == 0) part[warp] = make_float2(wm, s);
    __syncthreads();
    if (tid == 0) {
        float M = -INFINITY, total = 0.f;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part[w].x);
        for (int w = 0; w < kWarps; ++w) total += part[w].x > -INFINITY ? part[w].y * exp_diff(part[w].x, M) : 0.f;
        A.sums[blockIdx.x] = make_float2(M, total);
    }
    select_n(S, A.n, mine, [&](unsigned bound, auto&& take) {
        const float b = unorder(bound);
#pragma unroll
        for (int p = 0; p < PACKS; ++p)
            if (top[p] >= b) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float v = x[p].get(i);
                    if (v >= b) take(order(v + 0.f), (unsigned)(first + (p * kThreads + tid) * VEC + i));
                }
            }
    });
    for (int i = tid; i < A.n; i += kThreads) A.best[(long long)blockIdx.x * A.n + i] = S.out[i];
}

__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamArgs A)
{
    __shared__ SelectSmem S;
    __shared__ float row_score[kMaxBeams], row_max[kMaxBeams], row_log[kMaxBeams];
    __shared__ int kind[kMaxBeams], rows_on[kMaxBeams], rows_done[kMaxBeams], n_on, n_done;  // beams that go on, and finished ones
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row0 = (long long)blockIdx.x * A.K;
    if (tid < A.K) {
        const float score = A.scores[row0 + tid];
        row_score[tid] = score;
        kind[tid] = !(score > -INFINITY) ? -1 : A.done && A.done[row0 + tid] ? 1 : 0;
    }
    __syncthreads();
    if (tid == 0) {
        int on = 0, ended = 0;
        for (int k = 0; k < A.K; ++k) {
            if (kind[k] == 0) rows_on[on++] = k;
            else if (kind[k] > 0) rows_done[ended++] = k;
        }
        n_on = on;
        n_done = ended;
    }
    __syncthreads();
    tc::grid_dep_wait();

    // A thread takes items that follow one another (whole lists, best first, so that its largest is a list's
    // best), and threads next to one another are in different warps, so that each beam's are spread over all warps.
    const int place = lane * kWarps + warp;
    const int per = A.splits * A.n, kept = n_on * per, total = kept + n_done;
    const u64* best = A.best + row0 * per;
    int carried = 0;
    for (int from = 0; from < total || from == 0;) {
        // as many items as the threads hold, with the n best of those before
        const int left = total - from, most = kThreads * kItems - carried, now = left < most ? left : most;
        const int q = (now + carried + kThreads - 1) / kThreads;
        u64 key[kItems];
        int row[kItems];
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int at = place * q + i;  // among this round's items: new ones, then the carried
            key[i] = 0;
            row[i] = -1;
            if (i < q && at < now + carried) {
                if (at >= now) {
                    key[i] = S.out[at - now];
                } else if (from + at < kept) {
                    const int r = (from + at) / per;
                    row[i] = rows_on[r];
                    key[i] = best[(long long)row[i] * per + (from + at - r * per)];
                } else {
                    const int k = rows_done[from + at - kept];
                    key[i] = key_of(order(row_score[k] + 0.f), (unsigned)k * (unsigned)A.V + (unsigned)A.pad);
                }
            }
        }
        if (from == 0) {
            for (int r = warp; r < n_on; r += kWarps) {  // a row's log-sum-exp
                const int k = rows_on[r];
                float m = -INFINITY, s = 0.f;
                for (int i = lane; i < A.splits; i += 32) {
                    const float2 p = A.sums[(row0 + k) * A.splits + i];
                    const float big = fmaxf(m, p.x);
                    s = (m > -INFINITY ? s * exp_diff(m, big) : 0.f) + (p.x > -INFINITY ? p.y * exp_diff(p.x, big) : 0.f);
                    m = big;
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) {
                    const float m2 = __shfl_xor_sync(kAll, m, o), s2 = __shfl_xor_sync(kAll, s, o), big = fmaxf(m, m2);
                    s = (m > -INFINITY ? s * exp_diff(m, big) : 0.f) + (m2 > -INFINITY ? s2 * exp_diff(m2, big) : 0.f);
                    m = big;
                }
                if (lane == 0) {
                    row_max[k] = m;
                    row_log[k] = logf(s);
                }
            }
        }
        if (tid < 2) S.count[tid] = 0;
        __syncthreads();  // the carried keys have been read, too
        unsigned mine = 0;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (row[i] >= 0 && key[i] != 0) {
                const int k = row[i];
                const float x = unorder((unsigned)(key[i] >> 32)), m = row_max[k];
                const float c = row_score[k] + ((x == m ? 0.f : x - m) - row_log[k]) + 0.f;
                key[i] = c > -INFINITY ? key_of(order(c), (unsigned)k * (unsigned)A.V + (0xffffffffu - (unsigned)key[i])) : 0;
            }
            mine = max(mine, (unsigned)(key[i] >> 32));
        }
        const int R = tops_of(A.n);
        warp_tops(mine, R, S.top + warp * R, lane);
        __syncthreads();
        select_n(S, A.n, mine, [&](unsigned bound, auto&& take) {
#pragma unroll
            for (int i = 0; i < kItems; ++i)
                if ((unsigned)(key[i] >> 32) >= bound) take((unsigned)(key[i] >> 32), 0xffffffffu - (unsigned)key[i]);
        });
        carried = A.n;
        from += now > 0 ? now : 1;
    }

    const long long at = (long long)blockIdx.x * A.n;
    if (tid < A.n) {
        int found = 0;
        for (int i = 0; i < A.n; ++i) found += S.out[i] != 0;
        unsigned flat;
        float c = -INFINITY;
        if (tid < found) {
            flat = 0xffffffffu - (unsigned)S.out[tid];
            c = unorder((unsigned)(S.out[tid] >> 32));
        } else {
            // the (tid - found)-th lowest index that is not among the found ones
            flat = tid - found;
            for (bool again = true; again;) {
                unsigned below = 0;
                for (int j = 0; j < found; ++j) below += 0xffffffffu - (unsigned)S.out[j] <= flat;
                again = flat != (unsigned)(tid - found) + below;
                flat = (unsigned)(tid - found) + below;
            }
        }
        const int k = flat / (unsigned)A.V;
        A.scores_out[at + tid] = c;
        A.parent[at + tid] = k;
        A.token[at + tid] = flat - (unsigned)k * (unsigned)A.V;
        if (A.src_slots) A.src_slots[at + tid] = A.slots[row0 + k];
    }
}

struct BeamPlan {
    int packs, seg, splits;
    size_t off_best, bytes;
};

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

int check(const beam_params_t* p)
{
    if (!p) return fail(GDN_ERR_INVALID_ARG, "beam_select: params is NULL");
    if (p->N < 0 || p->K < 1 || p->V < 1) return fail(GDN_ERR_INVALID_ARG, "beam_select: N must be >= 0, K and V >= 1");
    if (p->row_stride < p->V) return fail(GDN_ERR_INVALID_ARG, "beam_select: row_stride is below V");
    if (!known_dtype(p->dtype)) return fail(GDN_ERR_INVALID_ARG, "beam_select: unknown dtype");
    if (p->K > kMaxBeams || p->n_out > kMaxOut) return fail(GDN_ERR_UNSUPPORTED, "beam_select: more than 64 beams or outputs");
    if (p->V > INT_MAX / p->K || p->N > INT_MAX / (64 * p->K)) return fail(GDN_ERR_UNSUPPORTED, "beam_select: K V or N K is too large");
    if (p->n_out < 1 || p->n_out > p->K * p->V) return fail(GDN_ERR_INVALID_ARG, "beam_select: n_out must be 1 .. K V");
    return GDN_OK;
}

// Segments of 8 packs a thread; of fewer where that would leave SMs without one.
BeamPlan plan_of(const beam_params_t* p)
{
    BeamPlan pl{};
    const int vec = 16 / (int)elem_size(p->dtype);
    // a row may start vec - 1 elements into its first pack; segments of one size leave no small last one,
    // whose few threads would give a low bound
    const int64_t span = p->V + vec - 1;
    pl.packs = 8;
    while (pl.packs > 2 && p->N * p->K * ((span + pl.packs * vec * kThreads - 1) / (pl.packs * vec * kThreads)) < 4 * kNumSMs) pl.packs /= 2;
    const int64_t most = (int64_t)pl.packs * vec * kThreads;
    pl.splits = (int)((span + most - 1) / most);
    pl.seg = (int)((span + (int64_t)pl.splits * vec - 1) / ((int64_t)pl.splits * vec)) * vec;
    const size_t segs = (size_t)(p->N * p->K) * pl.splits;
    pl.off_best = (segs * sizeof(float2) + 15) / 16 * 16;
    pl.bytes = pl.off_best + segs * p->n_out * sizeof(u64);
    return pl;
}

template <typename T>
void launch_segments(const BeamArgs& A, int packs, unsigned ctas, cudaStream_t st)
{
    if (packs == 8) beam_segment_kernel<T, 8><<<ctas, kThreads, 0, st>>>(A);
    else if (packs == 4) beam_segment_kernel<T, 4><<<ctas, kThreads, 0, st>>>(A);
    else beam_segment_kernel<T, 2><<<ctas, kThreads, 0, st>>>(A);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" size_t beam_workspace_bytes(const beam_params_t* p) { return check(p) == GDN_OK ? plan_of(p).bytes : 0; }

extern "C" int beam_select(const beam_params_t* p, const void* logits, const float* scores, const uint8_t* done,
                           const int32_t* slots, float* scores_out, int32_t* parent, int32_t* token, int32_t* src_slots,
                           void* workspace, size_t workspace_bytes, void* stream)
{
    const int st = check(p);
    if (st != GDN_OK) return st;
    if (p->N == 0) return GDN_OK;
    if (done && (p->pad_token < 0 || p->pad_token >= p->V)) return fail(GDN_ERR_INVALID_ARG, "beam_select: pad_token outside [0, V)");
    if (!logits || !scores || !scores_out || !parent || !token || (src_slots && !slots))
        return fail(GDN_ERR_INVALID_ARG, "beam_select: NULL pointer");
    const size_t es = elem_size(p->dtype);
    if ((uintptr_t)logits % es || (uintptr_t)scores % 4 || (uintptr_t)slots % 4 || (uintptr_t)scores_out % 4 || (uintptr_t)parent % 4 ||
        (uintptr_t)token % 4 || (uintptr_t)src_slots % 4 || (uintptr_t)workspace % 16)
        return fail(GDN_ERR_INVALID_ARG, "beam_select: a pointer is not aligned to its element (the workspace to 16 bytes)");
    const BeamPlan pl = plan_of(p);
    if (!workspace || workspace_bytes < pl.bytes)
        return fail(GDN_ERR_WORKSPACE, "beam_select: workspace smaller than beam_workspace_bytes()");
    const size_t rows = (size_t)(p->N * p->K), n_o = (size_t)p->N * p->n_out * 4;
    const struct { const void* ptr; size_t n; } in[] = {{logits, ((rows - 1) * (size_t)p->row_stride + (size_t)p->V) * es}, {scores, rows * 4}, {done, rows}, {slots, rows * 4}};
    const struct { const void* ptr; size_t n; } out[] = {{scores_out, n_o}, {parent, n_o}, {token, n_o}, {src_slots, n_o}, {workspace, pl.bytes}};
    for (int i = 0; i < 5; ++i) {
        for (const auto& o : in)
            if (overlap(out[i].ptr, out[i].n, o.ptr, o.n)) return fail(GDN_ERR_ALIAS, "beam_select: an output or the workspace overlaps an input");
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].ptr, out[i].n, out[j].ptr, out[j].n)) return fail(GDN_ERR_ALIAS, "beam_select: outputs overlap");
    }
    if (rows * pl.splits > (size_t)INT_MAX || (size_t)p->K * pl.splits * p->n_out > (size_t)INT_MAX)
        return fail(GDN_ERR_UNSUPPORTED, "beam_select: too many segments for one launch");
    BeamArgs A{};
    A.logits = logits; A.scores = scores; A.done = done; A.slots = slots;
    A.scores_out = scores_out; A.parent = parent; A.token = token; A.src_slots = src_slots;
    A.sums = (float2*)workspace; A.best = (u64*)((char*)workspace + pl.off_best);
    A.row_stride = p->row_stride; A.K = (int)p->K; A.V = (int)p->V; A.splits = pl.splits; A.seg = pl.seg; A.n = p->n_out; A.pad = p->pad_token;
    cudaStream_t cs = (cudaStream_t)stream;
    const unsigned ctas = (unsigned)(rows * pl.splits);
    if (p->dtype == GDN_F32) launch_segments<float>(A, pl.packs, ctas, cs);
    else if (p->dtype == GDN_BF16) launch_segments<__nv_bfloat16>(A, pl.packs, ctas, cs);
    else launch_segments<__half>(A, pl.packs, ctas, cs);
    int e = (int)cudaGetLastError();
    if (!e) {
        // The join starts while the segments run and waits on the device for their end.
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)p->N);
        cfg.blockDim = dim3(kThreads);
        cfg.stream = cs;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = (int)cudaLaunchKernelEx(&cfg, beam_join_kernel, A);
    }
    return e ? cuda_fail(e, "beam_select launch") : GDN_OK;
}
