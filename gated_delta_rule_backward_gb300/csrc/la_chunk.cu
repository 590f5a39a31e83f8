// la_chunk.cu -- linear attention's chunked form (include/la.h): the core of la_internal.h, 128 tokens at a time, on
// the 5th-generation tensor cores.
//
// Mathematics.  With G the running sum of a chunk's log decays, the chunk's part of the core is dense:
//     out = co (cs P' Z + e^G X S^T),   P'[t][s] = e^(G_t - G_s) x_t . y_s for s <= t
//     S  <- e^(G_last) S + cs Z^T Y',   Y'[t] = e^(G_last - G_t) y_t
// A call backwards in time walks its tokens, and with them the tiles' rows, from the last one on, each token decaying by
// the gate of the one behind it; nothing else changes.
//
// One CTA owns a state (D x D, fp32, in registers: thread = row j and half of the columns) and walks the chunks of a
// sequence's segment.  All tiles are [token][column] in shared memory, in core matrices of 8 tokens x 8 columns; X, Y and Z arrive by
// asynchronous copies as they are stored.  Products with a contraction over columns read a tile K-major, those over
// tokens read the same bytes MN-major, so that nothing is transposed:
//     P  = X Y^T          128 x 128, K = D     X, Y as stored: exact
//     XS = X S^T          128 x D,   K = D     S as bf16 hi + lo in shared memory: 2 passes
//     O  = P' Z           128 x D,   K = 128   P' as bf16 hi + lo in TMEM (in P's columns): 2 passes
//     dS = Z^T Y'         D x D,     K = 128   Y' as bf16 hi + lo in shared memory: 2 passes
// hi + lo carries 16 significant bits (2^-16 relative); the accumulators and the state are fp32.
//
// Decays.  G is summed in fp64 and kept as two fp32 numbers, since what is needed are small differences of sums that
// may be large.  e^(G_t - G_s) of 32 x 32 blocks below the diagonal is the product of a row's and a column's factor
// against the block's last column (each at most 1 for decays); only the diagonal block takes an exponential an element.
//
// Long sequences, few heads: segments, as many a sequence and head as fill the SMs.  A first kernel leaves each segment's
// own contribution to the state (dS alone, summed in TMEM from the last chunk back, against the segment's end) and its decay; the second
// starts each segment from the sum of those before it.
#include "gdn_device.cuh"
#include "gdn_elem.cuh"
#include "gdn_launch.cuh"
#include "gdn_tc.cuh"
#include "la_internal.h"

namespace gdn {
namespace {

__device__ int g_la_chunk_bad, g_la_chunk_timeout;

constexpr int L = 128;                 // tokens of a chunk
constexpr int kThreads = 256;          // two warps a scheduler, so that a thread can hold half a state's row and a tile's
constexpr int kIssuer = 128;           // issues the products: its warp has the least to do (columns 64 .. of rows 0 .. 31 of P' are zeros)
constexpr int kMostSegments = 16;
constexpr uint32_t kColP = 0, kColO = 128, kColXS = 256, kColS = 384, kTmemCols = 512;

struct LaChunkArgs {
    LaRun run;
    float *states, *decays;  // [n_seq H][segments][D D]: the state before, then each segment's contribution but the last; [n_seq H][segments]
    int segments, per;       // per sequence; chunks of one
    int vec, vec_out;
};

// Bytes of shared memory.
template <int D>
struct Smem {
    static constexpr int tile = L * D * 2;
    static constexpr int x = 0, y = tile, z = 2 * tile, yh = 3 * tile, yl = 4 * tile;
    static constexpr int sh = 5 * tile, sl = sh + D * D * 2;
    static constexpr int g = sl + D * D * 2;  // five arrays of L floats, then barriers
    static constexpr int bars = g + 5 * L * 4, sums = bars + 64, bytes = sums + 64;
    static constexpr int z1 = sh;  // the first kernel's second Z
};
static_assert(Smem<128>::bytes <= kSmemPerCtaMax, "shared memory");

struct Gates {
    float *hi, *lo, *e, *w, *c;  // G; e^G; e^(G_last - G); e^(G of the block's last column - G)
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where the walk's token i lies, and how far the next one.
struct Walk {
    long long first;
    int step;
    __device__ __forceinline__ long long row(long long i) const { return first + step * i; }
};

// Rows i0 .. i0 + 127 of the walk, those from n on as zeros.  A warp's 32 units of 16 bytes are 8 rows of 4: 64 bytes
// of each row from memory, whole core matrices to shared memory (no bank twice).
template <int D>
__device__ __forceinline__ void load_tile(char* sm, int tile, const __nv_bfloat16* src, long long stride, const Walk& w, long long i0, int n, bool vec)
{
    const int tid = threadIdx.x;
#pragma unroll
    for (int u0 = 0; u0 < L * D / 8; u0 += 256) {
        const int u = u0 + tid, r = (u & 7) + 8 * ((u >> 3) / (D / 8)), kc = (u >> 3) % (D / 8);
        const bool real = r < n;
        const __nv_bfloat16* from = src + w.row(real ? i0 + r : i0) * stride + 8 * kc;
        const int at = tile + (u >> 3) * 128 + (u & 7) * 16;
        if (vec) cp_async16(tc::smem_addr(sm + at), from, real);
        else {
            Pack<__nv_bfloat16, 8> p;
#pragma unroll
            for (int e = 0; e < 8; ++e) p.x[e] = real ? from[e] : __float2bfloat16(0.f);
            *reinterpret_cast<uint4*>(sm + at) = *reinterpret_cast<const uint4*>(&p);
        }
    }
}

// The gate before the walk's token i enters (0 where there is none: rows from n on, and backwards the first).
__device__ __forceinline__ double load_gate(const LaRun& A, const Walk& w, int h, long long i, bool real)
{
    if (!real || (A.reverse && i == 0)) return 0.0;
    const float g = ld_any(A.g, (w.row(i) + A.reverse) * A.gs0 + h * A.gs1, A.gate_dtype);
    return g < kLaLeastGate ? (double)kLaLeastGate : (double)g;
}

// Inclusive sums over the first 128 threads, by warps; the sums of the warps before come from shared memory behind a barrier.
__device__ __forceinline__ double scan_warp(double x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Y' = w Y as bf16 hi and lo: units of 16 bytes, each lane 8 columns of one token.
template <int D>
__device__ __forceinline__ void decayed_keys(char* sm, int y, int yh, int yl, const float* w)
{
    const int tid = threadIdx.x;
#pragma unroll 4
    for (int u0 = 0; u0 < L * D / 8; u0 += 256) {
        const int u = u0 + tid, r = (u & 7) + 8 * ((u >> 3) / (D / 8)), at = (u >> 3) * 128 + (u & 7) * 16;
        const uint4 v = *reinterpret_cast<const uint4*>(sm + y + at);
        const f2 ww = pack2(w[r], w[r]);
        uint4 hi, lo;
        auto part = [&](uint32_t x, uint32_t& h, uint32_t& l) {
            const float2 p = unpack2(mul2(pack2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)), ww));
            tc::split_bf16x2(p.x, p.y, h, l);
        };
        part(v.x, hi.x, lo.x);
        part(v.y, hi.y, lo.y);
        part(v.z, hi.z, lo.z);
        part(v.w, hi.w, lo.w);
        *reinterpret_cast<uint4*>(sm + yh + at) = hi;
        *reinterpret_cast<uint4*>(sm + yl + at) = lo;
    }
}

// Products, by one thread.  K-major: rows of the tile are M or N, columns K; MN-major: columns are M or N, rows K.
template <int D>
__device__ __forceinline__ uint64_t k_major(uint32_t tile, int slice) { return tc::make_desc(tile + slice * 256, 128, D * 16); }
template <int D>
__device__ __forceinline__ uint64_t mn_major(uint32_t tile, int slice) { return tc::make_desc(tile + slice * D * 32, D * 16, 128); }
constexpr uint32_t kTransposedA = 1u << 15, kTransposedB = 1u << 16;

// dS (+)= Z^T Y'; slices of 16 tokens
template <int D>
__device__ __forceinline__ void issue_state(uint32_t tmem, uint32_t z, uint32_t yh, uint32_t yl, int slices, bool accumulate)
{
    constexpr uint32_t idesc = tc::idesc_bf16(D) | kTransposedA | kTransposedB;
    for (int s = 0; s < slices; ++s) {
        const uint64_t a = mn_major<D>(z, s);
        tc::mma_ss16(tmem + kColS, a, mn_major<D>(yh, s), idesc, accumulate || s > 0);
        tc::mma_ss16(tmem + kColS, a, mn_major<D>(yl, s), idesc, 1);
    }
}

__device__ __forceinline__ float exp_diff2(float ah, float al, float bh, float bl) { return expf((ah - bh) + (al - bl)); }

template <int N>
__device__ __forceinline__ void ld_cols(uint32_t at, float (&v)[N])
{
    static_assert(N % 32 == 0, "columns");
#pragma unroll
    for (int i = 0; i < N; i += 32) tc::ld32(at + i, *reinterpret_cast<float(*)[32]>(v + i));
}

// What both kernels begin with: barriers and tensor memory.
template <int BARS>
__device__ __forceinline__ uint32_t begin(uint64_t* bars)
{
    uint32_t* holder = reinterpret_cast<uint32_t*>(bars + 6);
    int* err = reinterpret_cast<int*>(bars + 7);
    if (threadIdx.x == 0) {
        for (int i = 0; i < BARS; ++i) tc::mbar_init(bars + i, 1);
        tc::mbar_fence_init();
        *err = 0;
    }
    if (threadIdx.x < 32) tc::tmem_alloc(holder, kTmemCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    return *holder;
}

__device__ __forceinline__ float* state_of(const LaChunkArgs& A, int D, int nh, int segment)
{
    return A.states + ((long long)nh * A.segments + segment) * D * D;
}

// A row's columns [c0, c0 + N) of a state in memory.
template <int D, int N>
__device__ __forceinline__ void load_state(float (&m)[N], const float* head, int j, int c0, bool transposed)
{
    if (!transposed) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(m + i) = *reinterpret_cast<const float4*>(head + j * D + c0 + i);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) m[i] = head[(c0 + i) * D + j];
    }
}
template <int D, int N>
__device__ __forceinline__ void store_state(const float (&m)[N], float* head, int j, int c0, bool transposed)
{
    if (!transposed) {
#pragma unroll
        for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(head + j * D + c0 + i) = *reinterpret_cast<const float4*>(m + i);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) head[(c0 + i) * D + j] = m[i];
    }
}

// The chunks [c0, c1) of segment `segment` of a sequence of `len` tokens; last: no segment follows.
struct Part {
    long long c0, c1;
    bool none, last;
};
__device__ __forceinline__ Part part_of(const LaChunkArgs& A, long long len, int segment)
{
    const long long chunks = (len + L - 1) / L;
    Part p;
    p.c0 = (long long)segment * A.per;
    p.none = segment > 0 && p.c0 >= chunks;
    p.c1 = p.c0 + A.per < chunks ? p.c0 + A.per : chunks;
    p.last = p.c1 >= chunks;
    return p;
}

// Segment contributions: segments - 1 CTAs a sequence and head.
template <int D>
__global__ void __launch_bounds__(kThreads, 1) la_segment_kernel(const LaChunkArgs A)
{
    using S = Smem<D>;
    extern __shared__ __align__(128) char sm[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::bars);
    double* sums = reinterpret_cast<double*>(sm + S::sums);
    float* sw = reinterpret_cast<float*>(sm + S::g);
    volatile int& s_err = *reinterpret_cast<int*>(bars + 7);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per_seq = A.segments - 1, nh = blockIdx.x / per_seq, segment = blockIdx.x - nh * per_seq;
    const int n = nh / A.run.H, h = nh - n * A.run.H;
    begin_after();
    const LaSequence q = la_sequence(A.run, n);
    if (!q.ok) return;  // the second kernel reports it
    const long long len = q.hi - q.lo;
    const Part part = part_of(A, len, segment);
    if (part.none || part.last) return;
    const Walk w = {A.run.reverse ? q.hi - 1 : q.lo, A.run.reverse ? -1 : 1};
    const uint32_t tmem = begin<1>(bars);
    const __nv_bfloat16* y = (const __nv_bfloat16*)A.run.y + (h % A.run.yh) * A.run.ys1;
    const __nv_bfloat16* z = (const __nv_bfloat16*)A.run.z + (h % A.run.zh) * A.run.zs1;
    const uint32_t base = tc::smem_addr(sm);
    const int zt[2] = {S::z, S::z1};
    double carry = 0.0;
    const long long count = part.c1 - part.c0;
    bool fine = true;
    load_tile<D>(sm, S::y, y, A.run.ys0, w, (part.c1 - 1) * L, L, A.vec);
    load_tile<D>(sm, zt[0], z, A.run.zs0, w, (part.c1 - 1) * L, L, A.vec);
    cp_commit();
    for (long long it = 0; it < count; ++it) {
        const long long c = part.c1 - 1 - it;  // whole chunks: the sequence's last one is the last segment's
        double G = 0.0;
        if (tid < L) {
            G = scan_warp(load_gate(A.run, w, h, c * L + tid, true), lane);
            if (lane == 31) sums[warp] = G;
        }
        cp_wait<0>();
        __syncthreads();
        if (tid < L) {
            double all = 0.0;
            for (int i = 0; i < 4; ++i) {
                if (i < warp) G += sums[i];
                all += sums[i];
            }
            sw[tid] = expf((float)(carry + (all - G)));
        }
        for (int i = 0; i < 4; ++i) carry += sums[i];
        if (it > 0 && !tc::mbar_wait(bars, (uint32_t)(it - 1) & 1)) s_err = 1;  // the product before has read Y'
        __syncthreads();
        if (s_err) {
            fine = false;
            break;
        }
        decayed_keys<D>(sm, S::y, S::yh, S::yl, sw);
        tc::fence_async_smem();
        __syncthreads();
        if (it + 1 < count) {
            load_tile<D>(sm, S::y, y, A.run.ys0, w, (c - 1) * L, L, A.vec);
            load_tile<D>(sm, zt[(it + 1) & 1], z, A.run.zs0, w, (c - 1) * L, L, A.vec);
            cp_commit();
        }
        if (tid == kIssuer) {
            tc::fence_after();
            issue_state<D>(tmem, base + zt[it & 1], base + S::yh, base + S::yl, L / 16, it > 0);
            tc::commit(bars);
        }
    }
    cp_wait<0>();
    if (fine && !tc::mbar_wait(bars, (uint32_t)(count - 1) & 1)) s_err = 1;
    __syncthreads();
    if (s_err) {
        if (tid == 0) atomicOr(&g_la_chunk_timeout, 1);
    } else {
        tc::fence_after();
        const int j = 32 * (warp & 3) + lane, half = warp >> 2;
        float d[D / 2];
        ld_cols(tc::taddr(tmem, warp, kColS) + half * (D / 2), d);
        tc::wait_ld();
        if (j < D) {
#pragma unroll
            for (int i = 0; i < D / 2; ++i) d[i] *= A.run.cs;
            const float all = expf((float)carry);
            if (segment == 0) {
                // the state before it, kept for the segment's own start too (the last segment may replace it in place)
                float m[D / 2];
#pragma unroll
                for (int i = 0; i < D / 2; ++i) m[i] = 0.f;
                if (q.in >= 0) load_state<D>(m, A.run.s_in + q.in * A.run.in_stride + (long long)h * D * D, j, half * (D / 2), A.run.transposed_in);
                store_state<D>(m, state_of(A, D, nh, 0), j, half * (D / 2), false);
#pragma unroll
                for (int i = 0; i < D / 2; ++i) d[i] = fmaf(all, m[i], d[i]);
            }
            store_state<D>(d, state_of(A, D, nh, segment + 1), j, half * (D / 2), false);
            if (tid == 0) A.decays[nh * A.segments + segment + 1] = all;
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_free(tmem, kTmemCols);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) la_chunk_kernel(const LaChunkArgs A)
{
    using S = Smem<D>;
    constexpr int H = D / 2;  // columns of a thread
    extern __shared__ __align__(128) char sm[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::bars);
    uint64_t *bar_p = bars, *bar_xs = bars + 1, *bar_s = bars + 2, *bar_o = bars + 3;
    double* sums = reinterpret_cast<double*>(sm + S::sums);
    float* g0 = reinterpret_cast<float*>(sm + S::g);
    const Gates g = {g0, g0 + L, g0 + 2 * L, g0 + 3 * L, g0 + 4 * L};
    volatile int& s_err = *reinterpret_cast<int*>(bars + 7);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nh = blockIdx.x / A.segments, segment = blockIdx.x - nh * A.segments;
    const int n = nh / A.run.H, h = nh - n * A.run.H;
    begin_after();
    const LaSequence q = la_sequence(A.run, n);
    if (!q.ok) {
        if (tid == 0) atomicOr(&g_la_chunk_bad, 1);
        return;
    }
    const long long len = q.hi - q.lo;
    const Part part = part_of(A, len, segment);
    if (part.none) return;
    const Walk w = {A.run.reverse ? q.hi - 1 : q.lo, A.run.reverse ? -1 : 1};
    const uint32_t tmem = begin<4>(bars);
    const __nv_bfloat16* x = (const __nv_bfloat16*)A.run.x + (h % A.run.xh) * A.run.xs1;
    const __nv_bfloat16* y = (const __nv_bfloat16*)A.run.y + (h % A.run.yh) * A.run.ys1;
    const __nv_bfloat16* z = (const __nv_bfloat16*)A.run.z + (h % A.run.zh) * A.run.zs1;
    const uint32_t base = tc::smem_addr(sm);
    const bool vec = A.vec;
    const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;  // of TMEM: a chunk's token, or a state's row
    const bool has_state = row < D;
    auto tokens = [&](long long c) { return (int)(len - c * L < L ? len - c * L : L); };

    if (part.c0 < part.c1) {
        const int nt = tokens(part.c0);
        load_tile<D>(sm, S::x, x, A.run.xs0, w, part.c0 * L, nt, vec);
        load_tile<D>(sm, S::y, y, A.run.ys0, w, part.c0 * L, nt, vec);
        cp_commit();
        load_tile<D>(sm, S::z, z, A.run.zs0, w, part.c0 * L, nt, vec);
        cp_commit();
    }
    float m[H];
#pragma unroll
    for (int i = 0; i < H; ++i) m[i] = 0.f;
    if (has_state) {
        if (segment > 0) {
            for (int s = 1; s <= segment; ++s) {
                float d[H];
                const float a = s > 1 ? A.decays[nh * A.segments + s] : 0.f;
                load_state<D>(d, state_of(A, D, nh, s), row, half * H, false);
#pragma unroll
                for (int i = 0; i < H; ++i) m[i] = s > 1 ? fmaf(a, m[i], d[i]) : d[i];
            }
        } else if (!part.last) {
            load_state<D>(m, state_of(A, D, nh, 0), row, half * H, false);
        } else if (q.in >= 0) {
            load_state<D>(m, A.run.s_in + q.in * A.run.in_stride + (long long)h * D * D, row, half * H, A.run.transposed_in);
        }
    }
    auto put_state = [&]() {
#pragma unroll
        for (int i = 0; i < H; i += 8) {
            uint4 hi, lo;
            tc::split_bf16x2(m[i], m[i + 1], hi.x, lo.x);
            tc::split_bf16x2(m[i + 2], m[i + 3], hi.y, lo.y);
            tc::split_bf16x2(m[i + 4], m[i + 5], hi.z, lo.z);
            tc::split_bf16x2(m[i + 6], m[i + 7], hi.w, lo.w);
            const int at = ((row >> 3) * (D / 8) + (half * H + i) / 8) * 128 + (row & 7) * 16;
            *reinterpret_cast<uint4*>(sm + S::sh + at) = hi;
            *reinterpret_cast<uint4*>(sm + S::sl + at) = lo;
        }
    };
    if (has_state) put_state();

    bool fine = true;
    for (long long c = part.c0; c < part.c1; ++c) {
        const uint32_t phase = (uint32_t)(c - part.c0) & 1;
        const int nt = tokens(c), slices = (nt + 15) / 16, ahead = c + 1 < part.c1 ? tokens(c + 1) : 0;
        double G = 0.0;
        cp_wait<1>();  // X and Y
        tc::fence_async_smem();
        tc::fence_before();
        __syncthreads();
        if (tid == kIssuer) {
            tc::fence_after();
            for (int s = 0; s < D / 16; ++s) tc::mma_ss16(tmem + kColP, k_major<D>(base + S::x, s), k_major<D>(base + S::y, s), tc::idesc_bf16(L), s > 0);
            tc::commit(bar_p);
            for (int s = 0; s < D / 16; ++s) {
                const uint64_t a = k_major<D>(base + S::x, s);
                tc::mma_ss16(tmem + kColXS, a, k_major<D>(base + S::sh, s), tc::idesc_bf16(D), s > 0);
                tc::mma_ss16(tmem + kColXS, a, k_major<D>(base + S::sl, s), tc::idesc_bf16(D), 1);
            }
            tc::commit(bar_xs);
        }
        if (tid < L) {
            G = scan_warp(load_gate(A.run, w, h, c * L + tid, tid < nt), lane);
            if (lane == 31) sums[warp] = G;
        }
        __syncthreads();
        if (tid < L) {
            double all = 0.0, before = 0.0;
            for (int i = 0; i < 4; ++i) {
                if (i < warp) before += sums[i];
                all += sums[i];
            }
            const double end = before + sums[warp];  // of this block of 32
            G += before;
            g.hi[tid] = (float)G;
            g.lo[tid] = (float)(G - (double)g.hi[tid]);
            g.e[tid] = expf((float)G);
            g.w[tid] = expf((float)(all - G));
            g.c[tid] = expf((float)(end - G));
        }
        __syncthreads();
        decayed_keys<D>(sm, S::y, S::yh, S::yl, g.w);
        cp_wait<0>();  // Z
        tc::fence_async_smem();
        __syncthreads();
        if (tid == kIssuer) {
            tc::fence_after();
            issue_state<D>(tmem, base + S::z, base + S::yh, base + S::yl, slices, false);
            tc::commit(bar_s);
        }
        {
            if (!tc::mbar_wait(bar_p, phase)) s_err = 1;
            tc::fence_after();
            if (ahead) load_tile<D>(sm, S::y, y, A.run.ys0, w, (c + 1) * L, ahead, vec);
            // P' in the place of P: 32 columns at a time, hi and lo
            uint32_t ph[32], pl[32];
            const float gh = g.hi[row], gl = g.lo[row];
            const uint32_t from = tc::taddr(tmem, warp, kColP) + half * 64;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int block = 2 * half + b;
                if (block > quarter) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) ph[16 * b + i] = pl[16 * b + i] = 0u;
                } else {
                    float p[32];
                    tc::ld32(from + 32 * b, p);
                    const float rf = block < quarter ? exp_diff2(gh, gl, g.hi[32 * block + 31], g.lo[32 * block + 31]) : 0.f;
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const int s = 32 * block + i;
                        if (block < quarter) {
                            p[i] = p[i] * (rf * g.c[s]);
                            p[i + 1] = p[i + 1] * (rf * g.c[s + 1]);
                        } else {
                            p[i] = i <= lane ? p[i] * exp_diff2(gh, gl, g.hi[s], g.lo[s]) : 0.f;
                            p[i + 1] = i + 1 <= lane ? p[i + 1] * exp_diff2(gh, gl, g.hi[s + 1], g.lo[s + 1]) : 0.f;
                        }
                        tc::split_bf16x2(p[i], p[i + 1], ph[16 * b + i / 2], pl[16 * b + i / 2]);
                    }
                }
            }
            // both halves of these 32 rows have been read
            asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
            tc::st32(tc::taddr(tmem, warp, kColP) + half * 32, ph);
            tc::st32(tc::taddr(tmem, warp, kColP) + 64 + half * 32, pl);
            tc::wait_st();
        }
        tc::fence_before();
        __syncthreads();
        if (s_err) {
            fine = false;
            break;
        }
        if (tid == kIssuer) {
            tc::fence_after();
            constexpr uint32_t idesc = tc::idesc_bf16(D) | kTransposedB;
            for (int s = 0; s < slices; ++s) {
                const uint64_t b = mn_major<D>(base + S::z, s);
                tc::mma_ts16(tmem + kColO, tmem + kColP + 8 * s, b, idesc, s > 0);
                tc::mma_ts16(tmem + kColO, tmem + kColP + 64 + 8 * s, b, idesc, 1);
            }
            tc::commit(bar_o);
        }
        {
            if (!tc::mbar_wait(bar_xs, phase)) s_err = 1;
            if (ahead) load_tile<D>(sm, S::x, x, A.run.xs0, w, (c + 1) * L, ahead, vec);
            cp_commit();
            if (!tc::mbar_wait(bar_s, phase)) s_err = 1;
            tc::fence_after();
            {
                float d[H];
                ld_cols(tc::taddr(tmem, warp, kColS) + half * H, d);
                const float a = g.e[L - 1];
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < H; ++i) m[i] = fmaf(A.run.cs, d[i], a * m[i]);
            }
            if (has_state) put_state();
            if (!tc::mbar_wait(bar_o, phase)) s_err = 1;
            tc::fence_after();
            if (ahead) load_tile<D>(sm, S::z, z, A.run.zs0, w, (c + 1) * L, ahead, vec);
            cp_commit();
            float o[H], xs[H];
            ld_cols(tc::taddr(tmem, warp, kColO) + half * H, o);
            ld_cols(tc::taddr(tmem, warp, kColXS) + half * H, xs);
            const float c1 = A.run.co * A.run.cs, c2 = A.run.co * g.e[row];
            tc::wait_ld();
            if (row < nt) {
                const long long at = (w.row(c * L + row) * A.run.H + h) * D + half * H;
#pragma unroll
                for (int i = 0; i < H; ++i) o[i] = fmaf(c2, xs[i], c1 * o[i]);
                if (A.vec_out && A.run.out_dtype == GDN_BF16) {
#pragma unroll
                    for (int i = 0; i < H; i += 8)
                        *reinterpret_cast<uint4*>((__nv_bfloat16*)A.run.out + at + i) =
                            make_uint4(tc::pack_bf16x2(o[i], o[i + 1]), tc::pack_bf16x2(o[i + 2], o[i + 3]), tc::pack_bf16x2(o[i + 4], o[i + 5]), tc::pack_bf16x2(o[i + 6], o[i + 7]));
                } else if (A.vec_out && A.run.out_dtype == GDN_F32) {
#pragma unroll
                    for (int i = 0; i < H; i += 4) *reinterpret_cast<float4*>((float*)A.run.out + at + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < H; ++i) st_any(A.run.out, at + i, A.run.out_dtype, o[i]);
                }
            }
        }
    }
    cp_wait<0>();
    tc::fence_before();
    __syncthreads();
    if (s_err) fine = false;
    if (!fine) {
        if (tid == 0) atomicOr(&g_la_chunk_timeout, 1);
    } else if (has_state && part.last && q.out >= 0) {
        if (A.run.reverse && len > 0) {
            const float a = expf(ld_any(A.run.g, q.lo * A.run.gs0 + h * A.run.gs1, A.run.gate_dtype));
#pragma unroll
            for (int i = 0; i < H; ++i) m[i] *= a;
        }
        store_state<D>(m, A.run.s_out + q.out * A.run.out_stride + (long long)h * D * D, row, half * H, A.run.transposed_out);
    }
    if (warp == 0) tc::tmem_free(tmem, kTmemCols);
}

// Segments a sequence and head: as many as leave every SM one, each of several chunks.
void plan(const LaRun& A, int* segments, int* per)
{
    const long long heads = (long long)A.n_seq * A.H;
    const long long chunks = ((long long)A.T + L - 1) / L;
    long long s = heads > 0 ? kNumSMs / heads : 1;
    if (s > kMostSegments) s = kMostSegments;
    if (s > chunks) s = chunks;
    if (s < 1) s = 1;
    const long long p = chunks > 0 ? (chunks + s - 1) / s : 1;
    *per = (int)p;
    *segments = (int)(chunks > 0 ? (chunks + p - 1) / p : 1);
}

bool vec16(const void* ptr, long long s0, long long s1) { return (uintptr_t)ptr % 16 == 0 && s0 % 8 == 0 && s1 % 8 == 0; }

template <int D>
int launch(const LaChunkArgs& A, cudaStream_t st)
{
    int e = (int)cudaFuncSetAttribute(la_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::bytes);
    if (!e && A.segments > 1) {
        e = (int)cudaFuncSetAttribute(la_segment_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::bytes);
        if (!e) e = launch_after(la_segment_kernel<D>, (unsigned)(A.run.n_seq * A.run.H * (A.segments - 1)), kThreads, Smem<D>::bytes, st, A);
    }
    if (!e) e = launch_after(la_chunk_kernel<D>, (unsigned)(A.run.n_seq * A.run.H * A.segments), kThreads, Smem<D>::bytes, st, A);
    return e;
}

}  // namespace

bool la_chunk_fits(const la_params_t* p)
{
    return p->in_dtype == GDN_BF16 && p->S_k == p->S_v && (p->S_k == 64 || p->S_k == 128) && p->T >= 32;
}

size_t la_chunk_workspace(const LaRun& A)
{
    int segments, per;
    plan(A, &segments, &per);
    return segments > 1 ? (size_t)A.n_seq * A.H * segments * ((size_t)A.DK * A.DV + 1) * sizeof(float) : 0;
}

int launch_la_chunk(const LaRun& run, void* workspace, cudaStream_t st)
{
    LaChunkArgs A{};
    A.run = run;
    plan(run, &A.segments, &A.per);
    A.states = (float*)workspace;
    A.decays = A.states + (long long)run.n_seq * run.H * A.segments * run.DK * run.DV;
    A.vec = vec16(run.x, run.xs0, run.xs1) && vec16(run.y, run.ys0, run.ys1) && vec16(run.z, run.zs0, run.zs1);
    A.vec_out = (uintptr_t)run.out % 16 == 0;
    return run.DK == 128 ? launch<128>(A, st) : launch<64>(A, st);
}

int la_chunk_take_bad(void* stream, int* status) { return la_take_word(&g_la_chunk_bad, stream, status); }
int la_chunk_take_timeout(void* stream, int* status) { return la_take_word(&g_la_chunk_timeout, stream, status); }

}  // namespace gdn
