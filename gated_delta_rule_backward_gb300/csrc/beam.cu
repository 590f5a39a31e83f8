// beam.cu -- a beam search's selection over beams and vocabulary (include/beam.h).
//
// Two kernels.  The first cuts every beam's row into segments, one a CTA, and reads each once:
// every 1 to 32 threads leave the maximum of their share (a chunk: their packs of 16 bytes),
// every CTA its maximum and the sum of exponentials against it.  The second, one CTA a sequence, joins the sums
// into each row's log-sum-exp, turns chunk maxima into scores, and looks at the few chunks alone that can
// hold one of the n best: an element among them is at least the n-th largest chunk maximum.
//
// The n-th largest chunk maximum is found in two steps.  The largest that n of the warps' few
// largest thread maxima reach is a bound that n chunks reach at least, and for chunks in no
// particular order few more do; those go to a list, and each listed chunk that fewer than n
// others exceed is read again.  Elements that reach the last of these go to a list of their own,
// and each one's rank is the number of listed keys above its own.  Keys are (score, lowest
// index first) in one 64-bit number, so ranks do not depend on the lists' order.  Where a list
// does not hold all that reach the bound (very many equal scores), n rounds of a CTA-wide
// maximum over the chunks that reach it select instead: right, but as slow as n readings of a sequence's rows
// by one CTA (16 x 8 rows of 128257 equal logits 1.3 ms; with all but three tokens next to each other at the type's lowest value, 4.3 ms).
//
// The stream is bound by the exponentials' instructions (eight a logit with the maximum) and, for few
// rows, by latency: 16 x 8 rows of 128257 bf16 logits 13.4 us in a graph, join and all, 128 x 8 rows of 151937 64 us,
// 4.9 TB/s.  Selecting inside every segment instead (a list and its ranks a CTA) took 17 us for the stream.
// The join is a chain of loads and barriers: what it runs is kept short and free of branches (the 16 x 8 rows
// took 15.7 us in a graph before that and the wider stream loads).  Its first loads, of scores and finished beams, wait
// for the stream too: 0.3 to 0.7 us a call.
#include <climits>
#include <cstdio>
#include <type_traits>

#include "../../include/beam.h"
#include "gdn_elem.cuh"
#include "gdn_f32x2.cuh"
#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_packs.h"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;           // of a segment
constexpr int kJoinThreads = 512, kJoinWarps = kJoinThreads / 32;
constexpr int kMaxOut = 64, kMaxBeams = 64;
constexpr int kList = 1024;  // items a list holds
constexpr int kFew = 32;     // chunks that are read without a closer bound
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
    float2* sums;   // [N K][splits] maximum and sum of a segment
    float* chunks;  // [N K][splits][kThreads >> lg] the maximum of 1 << lg threads
    long long row_stride;
    int K, V, splits, seg, lg_packs, lg, n, pad;
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

// A row's packs lie on 16-byte boundaries: it starts `lead` elements into the first.  Pack p of thread t of segment
// `split` begins at element split seg - lead + (256 p + t) VEC; what is outside the row or the segment reads as -inf.
template <typename T>
struct Segment {
    const T* at;  // on 16 bytes
    unsigned column;  // of its first element, in unsigned arithmetic (the first segment may begin before the row)
    int lo, end;
};
template <typename T>
__device__ __forceinline__ Segment<T> segment_of(const BeamArgs& A, const T* row, int split)
{
    const unsigned lead = (unsigned)(((uintptr_t)row & 15) / sizeof(T));
    const PackSegment s = pack_segment((unsigned)split, A.seg, lead, A.V);
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

// PACKS loads of 16 bytes a thread.
template <typename T, int PACKS>
__global__ void __launch_bounds__(kThreads, 4) beam_segment_kernel(const BeamArgs A)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    __shared__ float2 part[kWarps];
    const int row = blockIdx.x / A.splits, split = blockIdx.x - row * A.splits;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    begin_after();
    const T* base = (const T*)A.logits + row * A.row_stride;
    if ((A.done && A.done[row]) || !(A.scores[row] > -INFINITY)) return;

    Pack<T, VEC> x[PACKS];
    ld_chunk_packs<T, VEC, PACKS>(x, segment_of(A, base, split), [&](int p) { return (p * kThreads + tid) * VEC; });
    float m = -INFINITY;
#pragma unroll
    for (int p = 0; p < PACKS; ++p) m = fmaxf(m, pack_max(x[p]));  // a pack of NaNs: -inf stays
    // The sum against the thread's own maximum, 2^((x - m) L) with L = log2 e, as 2^(x L - r) for r = m L rounded: one
    // product and sum an element, and what r is off by is taken out of the sum at the end.
    float s = 0.f;
    if (m < INFINITY && m > -INFINITY) {
        const float r = m * kLog2e;
        const f2 rr = pack2(-r, -r), ll = pack2(kLog2e, kLog2e);
        f2 s2 = 0;
#pragma unroll
        for (int p = 0; p < PACKS; ++p)
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                const float2 v = unpack2(fma2(x[p].pair(i), ll, rr));
                s2 = add2(s2, pack2(ex2(v.x), ex2(v.y)));
            }
        s = sum2(s2) * ex2(-fmaf(m, kLog2e, -r));
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
    float cm = m;
    for (int o = 1; o < 1 << A.lg; o <<= 1) cm = fmaxf(cm, __shfl_xor_sync(kAll, cm, o));
    if ((lane & ((1 << A.lg) - 1)) == 0) A.chunks[((long long)blockIdx.x * kThreads + tid) >> A.lg] = cm;
    const float wm = unorder(__reduce_max_sync(kAll, order(m + 0.f)));
    s = m > -INFINITY ? s * exp_diff(m, wm) : 0.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    if (lane == 0) part[warp] = make_float2(wm, s);
    __syncthreads();
    if (tid == 0) {
        float M = -INFINITY, total = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part[w].x);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) total += part[w].x > -INFINITY ? part[w].y * exp_diff(part[w].x, M) : 0.f;
        A.sums[blockIdx.x] = make_float2(M, total);
    }
}

// Thread maxima that a warp of the join gives for a bound on the n-th: 32 or 64 in all.
__device__ __forceinline__ int tops_of(int n) { return (n <= 16 ? 32 : 64) / kJoinWarps; }

// The largest of the tops that n of them reach, by one warp.
__device__ __forceinline__ unsigned nth_top(const unsigned* top, int n, int lane)
{
    const uint4* all = reinterpret_cast<const uint4*>(top);
    const int tops = tops_of(n) * kJoinWarps;
    unsigned best = 0;
    for (int at = lane; at < tops; at += 32) {
        const unsigned v = top[at];
        int reach = 0;
#pragma unroll 4
        for (int i = 0; i < tops / 4; ++i) {
            const uint4 t = all[i];
            reach += (t.x >= v) + (t.y >= v) + (t.z >= v) + (t.w >= v);
        }
        if (reach >= n) best = max(best, v);
    }
    best = __reduce_max_sync(kAll, best);
    return best > kNegInf ? best : kNegInf + 1;  // an item at -inf is none
}

constexpr int kMostReads = 8;  // packs of a chunk that a thread has in flight
constexpr int kHeld = 2;  // chunks whose maxima a thread of the join keeps in registers

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const BeamArgs A)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    __shared__ u64 list[2][kList];
    __shared__ u64 out[kMaxOut], warp_best[kJoinWarps];
    __shared__ __align__(16) unsigned top[64];
    __shared__ float row_score[kMaxBeams], row_max[kMaxBeams], row_log[kMaxBeams];
    __shared__ int kind[kMaxBeams], rows_on[kMaxBeams], row_slot[kMaxBeams], n_on, chunk_count, element_count, kept_count;
    __shared__ unsigned the_bound, least_kept;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row0 = (long long)blockIdx.x * A.K;
    const int per = A.splits * (kThreads >> A.lg);  // chunks of a row
    // The wait comes before the scores too, although the segments' kernel has waited for whoever wrote those: it made
    // them visible to itself alone.
    begin_after();
    if (tid < A.K) {
        const float score = A.scores[row0 + tid];
        row_score[tid] = score;
        row_slot[tid] = A.src_slots ? A.slots[row0 + tid] : 0;
        kind[tid] = !(score > -INFINITY) ? -1 : A.done && A.done[row0 + tid] ? 1 : 0;
    }
    if (tid == 0) {
        chunk_count = element_count = kept_count = 0;
        least_kept = 0xffffffffu;
    }
    __syncthreads();
    if (warp == 0) {  // the beams that go on, in order
        int on = 0;
        for (int k0 = 0; k0 < A.K; k0 += 32) {
            const bool goes = k0 + lane < A.K && kind[k0 + lane] == 0;
            const unsigned all = __ballot_sync(kAll, goes);
            if (goes) rows_on[on + __popc(all & ((1u << lane) - 1))] = k0 + lane;
            on += __popc(all);
        }
        if (lane == 0) n_on = on;
    }
    __syncthreads();
    const int all_chunks = n_on * per;
    // A thread's chunks are tid + j kJoinThreads of the going beams' chunks; the first kHeld stay in registers.
    float held[kHeld];
    int held_row[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int i = tid + j * kJoinThreads;
        held[j] = -INFINITY;
        held_row[j] = 0;
        if (i < all_chunks) {
            const int r = i / per;
            held_row[j] = rows_on[r];
            held[j] = __ldcg(A.chunks + (row0 + held_row[j]) * per + (i - r * per));
        }
    }
    for (int r = warp; r < n_on; r += kJoinWarps) {  // a row's log-sum-exp
        const int k = rows_on[r];
        float m = -INFINITY, s = 0.f;
        for (int i = lane; i < A.splits; i += 32) {
            const float2 p = A.sums[(row0 + k) * A.splits + i];
            const float big = fmaxf(m, p.x);
            s = (m > -INFINITY ? s * exp_diff(m, big) : 0.f) + (p.x > -INFINITY ? p.y * exp_diff(p.x, big) : 0.f);
            m = big;
        }
        const float big = unorder(__reduce_max_sync(kAll, order(m + 0.f)));
        s = m > -INFINITY ? s * exp_diff(m, big) : 0.f;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        if (lane == 0) {
            row_max[k] = big;
            row_log[k] = logf(s);
        }
    }
    __syncthreads();

    // order(score) of a beam's logit; 0 for one that is none
    struct Beam {
        float score, max, log;
        __device__ __forceinline__ unsigned of(float x) const
        {
            const float c = score + ((x == max ? 0.f : x - max) - log) + 0.f;  // + 0: -0 becomes 0
            const unsigned o = order(c);
            return (x > -INFINITY) & (c > -INFINITY) ? o : 0u;
        }
    };
    auto beam_of = [&](int k) { return Beam{row_score[k], row_max[k], row_log[k]}; };
    // every chunk of this thread: (its number among the going beams' chunks, order(its maximum's score))
    auto each_chunk = [&](auto&& take) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) take(tid + j * kJoinThreads, beam_of(held_row[j]).of(held[j]));
        for (int i = tid + kHeld * kJoinThreads; i < all_chunks; i += kJoinThreads) {
            const int r = i / per, k = rows_on[r];
            take(i, beam_of(k).of(__ldcg(A.chunks + (row0 + k) * per + (i - r * per))));
        }
    };
    // every element of the going beams' chunk i that reaches `least`, shared by LC threads with `reads` packs in
    // flight each: (order(score), index)
    auto elements_of = [&](auto reads, int i, int LC, unsigned least, auto&& take) {
        constexpr int kReads = decltype(reads)::value;
        const int r = i / per, c = i - r * per, k = rows_on[r];
        const Beam beam = beam_of(k);
        const int split = c / (kThreads >> A.lg), t0 = (c - split * (kThreads >> A.lg)) << A.lg;
        const Segment<T> s = segment_of(A, (const T*)A.logits + (row0 + k) * A.row_stride, split);
        for (int q0 = tid & (LC - 1); q0 < 1 << (A.lg_packs + A.lg); q0 += kReads * LC) {
            Pack<T, VEC> x[kReads];
            auto in = [&](int p) {
                const int q = q0 + LC * p;
                return q < 1 << (A.lg_packs + A.lg) ? ((q >> A.lg) * kThreads + t0 + (q & ((1 << A.lg) - 1))) * VEC : A.seg;
            };
            ld_chunk_packs<T, VEC, kReads>(x, s, in);
            unsigned reach = 0;  // the packs that hold such an element: few, so they are read again one by one
#pragma unroll
            for (int p = 0; p < kReads; ++p) reach |= (beam.of(pack_max(x[p])) >= least ? 1u : 0u) << p;
#pragma unroll 1
            for (; reach; reach &= reach - 1) {
                const int one = in(__ffs(reach) - 1);
                Pack<T, VEC> y[1];
                ld_chunk_packs<T, VEC, 1>(y, s, [&](int) { return one; });
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const unsigned o = beam.of(y[0].get(e));
                    if (o >= least) take(o, (unsigned)k * (unsigned)A.V + (s.column + (unsigned)(one + e)));
                }
            }
        }
    };

    auto each_element = [&](int i, int LC, unsigned least, auto&& take) {
        if (1 << (A.lg_packs + A.lg) <= LC) elements_of(std::integral_constant<int, 1>(), i, LC, least, take);
        else elements_of(std::integral_constant<int, kMostReads>(), i, LC, least, take);
    };

    unsigned mine = 0;
    each_chunk([&](int, unsigned o) { mine = max(mine, o); });
    {
        unsigned v = mine;
        const int R = tops_of(A.n);
        for (int r = 0; r < R; ++r) {
            const unsigned best = __reduce_max_sync(kAll, v);
            if (lane == 0) top[warp * R + r] = best;
            const unsigned who = __ballot_sync(kAll, v == best);
            if (lane == __ffs(who) - 1) v = 0;
        }
    }
    __syncthreads();
    if (warp == 0) {
        const unsigned b = nth_top(top, A.n, lane);
        if (lane == 0) the_bound = b;
    }
    __syncthreads();
    const unsigned bound = the_bound;
    if (mine >= bound)
        each_chunk([&](int i, unsigned o) {
            if (o >= bound) {
                const int at = atomicAdd(&chunk_count, 1);
                if (at < kList) list[0][at] = key_of(o, (unsigned)i);
            }
        });
    __syncthreads();
    const int chunks = chunk_count;
    bool fits = chunks <= kList;
    int found = 0;  // candidates above -inf among the n best
    unsigned least = bound;  // what an element has to reach
    if (fits) {
        const u64* chunk = list[0];
        int kept = chunks;
        u64* elements = list[1];
        if (chunks > kFew && chunks > A.n) {
            // the chunks that fewer than n others exceed, and with them a closer bound
            for (int t = tid; t < chunks; t += kJoinThreads) {
                const unsigned v = (unsigned)(list[0][t] >> 32);
                int above = 0;
                for (int i = 0; i < chunks; ++i) above += (unsigned)(list[0][i] >> 32) > v;
                if (above < A.n) {
                    list[1][atomicAdd(&kept_count, 1)] = list[0][t];
                    atomicMin(&least_kept, v);
                }
            }
            __syncthreads();
            kept = kept_count;
            least = least_kept;
            chunk = list[1];
            elements = list[0];
        }
        auto push = [&](unsigned o, unsigned index) {
            const int at = atomicAdd(&element_count, 1);
            if (at < kList) elements[at] = key_of(o, index);
        };
        // a warp a chunk, or as many threads as there are for each
        int lg_lanes = 5;
        while (lg_lanes > 2 && kept << lg_lanes > kJoinThreads) --lg_lanes;
        for (int t = tid >> lg_lanes; t < kept; t += kJoinThreads >> lg_lanes)
            each_element((int)(0xffffffffu - (unsigned)chunk[t]), 1 << lg_lanes, least, push);
        if (tid < A.K && kind[tid] > 0 && order(row_score[tid] + 0.f) >= least) push(order(row_score[tid] + 0.f), (unsigned)tid * (unsigned)A.V + (unsigned)A.pad);
        __syncthreads();
        const int listed = element_count;
        fits = listed <= kList;
        if (fits) {
            found = listed < A.n ? listed : A.n;
            for (int t0 = 0; t0 < listed; t0 += kJoinThreads / 8) {  // eight threads a key
                const int t = t0 + tid / 8;
                const u64 key = t < listed ? elements[t] : ~0ull;
                int rank = 0;
                for (int i = tid & 7; i < listed; i += 8) rank += elements[i] > key;
#pragma unroll
                for (int o = 4; o >= 1; o >>= 1) rank += __shfl_xor_sync(kAll, rank, o);
                if (t < listed && (tid & 7) == 0 && rank < A.n) out[rank] = key;
            }
            __syncthreads();
        }
    }
    if (!fits) {
        found = 0;
        u64 last = ~0ull;
        for (int r = 0; r < A.n; ++r) {
            u64 best = 0;
            auto better = [&](unsigned o, unsigned index) {
                const u64 key = key_of(o, index);
                if (key < last && key > best) best = key;
            };
            for (int i = warp; i < all_chunks; i += kJoinWarps) {
                const int r = i / per, c = i - r * per, k = rows_on[r];
                if (beam_of(k).of(__ldcg(A.chunks + (row0 + k) * per + c)) >= bound) each_element(i, 32, max(bound, (unsigned)(best >> 32)), better);
            }
            if (tid < A.K && kind[tid] > 0) better(order(row_score[tid] + 0.f), (unsigned)tid * (unsigned)A.V + (unsigned)A.pad);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) {
                const u64 other = __shfl_xor_sync(kAll, best, o);
                best = other > best ? other : best;
            }
            if (lane == 0) warp_best[warp] = best;
            __syncthreads();
            last = 0;
            for (int i = 0; i < kJoinWarps; ++i) last = warp_best[i] > last ? warp_best[i] : last;
            if (tid == 0) out[r] = last;
            found += last != 0;
            __syncthreads();
        }
    }

    const long long at = (long long)blockIdx.x * A.n;
    if (tid < A.n) {
        unsigned flat;
        float c = -INFINITY;
        if (tid < found) {
            flat = 0xffffffffu - (unsigned)out[tid];
            c = unorder((unsigned)(out[tid] >> 32));
        } else {
            // the (tid - found)-th lowest index that is not among the found ones
            flat = tid - found;
            for (bool again = true; again;) {
                unsigned below = 0;
                for (int j = 0; j < found; ++j) below += 0xffffffffu - (unsigned)out[j] <= flat;
                again = flat != (unsigned)(tid - found) + below;
                flat = (unsigned)(tid - found) + below;
            }
        }
        const int k = flat / (unsigned)A.V;
        A.scores_out[at + tid] = c;
        A.parent[at + tid] = k;
        A.token[at + tid] = flat - (unsigned)k * (unsigned)A.V;
        if (A.src_slots) A.src_slots[at + tid] = row_slot[k];
    }
}

struct BeamPlan {
    int lg_packs, seg, splits, lg;
    size_t off_chunks, bytes;
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
    // a row may start vec - 1 elements into its first pack; segments of one size leave no small last one
    const int64_t span = p->V + vec - 1;
    pl.lg_packs = 3;
    auto most = [&]() { return (int64_t)vec * kThreads << pl.lg_packs; };
    while (pl.lg_packs > 1 && p->N * p->K * ((span + most() - 1) / most()) < 4 * kNumSMs) --pl.lg_packs;
    pl.splits = (int)((span + most() - 1) / most());
    pl.seg = (int)((span + (int64_t)pl.splits * vec - 1) / ((int64_t)pl.splits * vec)) * vec;
    const size_t segs = (size_t)(p->N * p->K) * pl.splits;
    // chunks of up to 32 threads, as long as the join has kHeld for each of its threads
    const int64_t want = kHeld * kJoinThreads;
    while (pl.lg < 5 && p->K * pl.splits * (kThreads >> (pl.lg + 1)) >= want) ++pl.lg;
    pl.off_chunks = (segs * sizeof(float2) + 255) / 256 * 256;
    pl.bytes = pl.off_chunks + segs * (kThreads >> pl.lg) * sizeof(float);
    return pl;
}

template <typename T>
int launch_beam(const BeamArgs& A, unsigned segments, unsigned sequences, cudaStream_t st)
{
    const auto segment = A.lg_packs == 3 ? beam_segment_kernel<T, 8> : A.lg_packs == 2 ? beam_segment_kernel<T, 4> : beam_segment_kernel<T, 2>;
    const int e = launch_after(segment, segments, kThreads, 0, st, A);
    return e ? e : launch_after(beam_join_kernel<T>, sequences, kJoinThreads, 0, st, A);
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
    // chunks of a sequence are numbered in 32 bits
    if (rows * pl.splits > (size_t)INT_MAX || (size_t)p->K * pl.splits * kThreads > (size_t)INT_MAX)
        return fail(GDN_ERR_UNSUPPORTED, "beam_select: too many segments for one launch");
    BeamArgs A{};
    A.logits = logits; A.scores = scores; A.done = done; A.slots = slots;
    A.scores_out = scores_out; A.parent = parent; A.token = token; A.src_slots = src_slots;
    A.sums = (float2*)workspace; A.chunks = (float*)((char*)workspace + pl.off_chunks);
    A.row_stride = p->row_stride; A.K = (int)p->K; A.V = (int)p->V; A.splits = pl.splits; A.seg = pl.seg; A.lg_packs = pl.lg_packs; A.lg = pl.lg; A.n = p->n_out; A.pad = p->pad_token;
    cudaStream_t cs = (cudaStream_t)stream;
    const unsigned ctas = (unsigned)(rows * pl.splits);
    const int e = p->dtype == GDN_F32    ? launch_beam<float>(A, ctas, (unsigned)p->N, cs)
                  : p->dtype == GDN_BF16 ? launch_beam<__nv_bfloat16>(A, ctas, (unsigned)p->N, cs)
                                         : launch_beam<__half>(A, ctas, (unsigned)p->N, cs);
    return e ? cuda_fail(e, "beam_select launch") : GDN_OK;
}
