// la_chunk.cu -- linear attention's chunked form (include/la.h): the core of la_internal.h, 128 tokens at a time, on
// the 5th-generation tensor cores.
//
// Mathematics.  With G the running sum of a chunk's log decays, the chunk's part of the core is dense:
//     out = co (cs P' Z + e^G X S^T),   P'[t][s] = e^(G_t - G_s) x_t . y_s for s <= t
//     S  <- e^(G_last) S + cs Z^T Y',   Y'[t] = e^(G_last - G_t) y_t
// A call backwards in time walks its tokens, and with them the tiles' rows, from the last one on, each token decaying by
// the gate of the one behind it; nothing else changes.
//
// One CTA owns a state (D x D, fp32, transposed in TMEM) and walks the chunks of a
// sequence's segment.  X, Y and Z arrive by TMA as they are stored, rows of 64 columns in 128-byte swizzle.  Products with a
// contraction over columns read a tile K-major, those over tokens read the same bytes MN-major:
//     P   = X Y^T          128 x 128, K = D     X, Y as stored: exact
//     O   = X S^T          128 x D,   K = D     S as bf16 hi + lo in shared memory: 2 passes
//     O   <- e^G O + P' Z  128 x D,   K = 128   P' (with cs) as bf16 hi + lo in TMEM, in P's columns: 2 passes
//     S^T <- a S^T + Y'^T Z  D x D,   K = 128   Y'^T (with cs) as bf16 hi + lo in TMEM: 2 passes
// hi + lo carries 16 significant bits (2^-16 relative); the accumulators and the state are fp32.  What bounds the products, beside the tensor
// cores' own rate, is shared memory, which hands 128 bytes a cycle to all of them and the threads; so the operands that are made here are made in
// tensor memory, Y'^T by way of transposing loads.
//
// Groups of warps work on chunks side by side: eight turn P into P' and scale O's rows by e^G; eight make Y' and keep the state; four write the output.
// Four more serve them: one issues all products, in the order P, X S^T, dS, P' Z, so that no warp with work of its own stands in the
// products' queue; one issues all loads, one the stores of whole chunks; one sums the gates.  They meet at mbarriers only.  Loops over
// columns are rolled where registers allow: what the warps lacked most with all of it unrolled was instructions.
//
// Decays.  G is summed in 64-bit fixed point (powers of two, 31 fraction bits) and kept as a whole and a fractional fp32 number, since
// what is needed are small differences of sums that may be large.  e^(G_t - G_s) of 32 x 32 blocks off the diagonal is the product of a
// row's and a column's factor against the block's last column in walking order (each at most 1 for decays); only the diagonal block takes an
// exponential an element.
//
// Long sequences, few heads: segments, as many a sequence and head as fill the SMs.  A first kernel leaves each segment's
// own contribution to the state (dS alone, summed in TMEM from the last chunk back, against the segment's end) and its decay; the second
// starts each segment from the sum of those before it.
//
// Measured: a prompt of 4096 tokens, 48 heads of 128 (3 segments a head), 70 us; of 32768 tokens, 16 heads (9 segments), 174 us; 23
// prompts of up to 701 tokens, 16 heads, 60 us.  A chunk of 128 x 128 takes a CTA 3.0 us.  What bounds it is the chain of handovers from one chunk's state to the
// next and the shared memory that products and threads share: alone and cold, the first kernel 26 us and the second 52 for the 4096 tokens, tensor pipe
// 44 % of the second's time, issue slots 41 %, DRAM 27 %.
#include <cuda.h>

#include "gdn_device.cuh"
#include "gdn_elem.cuh"
#include "gdn_launch.cuh"
#include "gdn_tc.cuh"
#include "la_internal.h"

namespace gdn {
namespace {

__device__ int g_la_chunk_status[2];  // bad slots and token ranges; waits that gave up

constexpr int L = 128;         // tokens of a chunk
constexpr int kGroup = 256;    // threads of a group
constexpr int kThreads = 2 * kGroup + 256;
constexpr int kWriters = 16, kIssuer = 20, kLoader = 21, kSummer = 22, kStorer = 23;  // warps
constexpr int kMostSegments = 16;
constexpr uint32_t kColP = 0, kColO = 128, kColS = 256, kColY = 384, kTmemCols = 512;  // Y': 64 columns of hi words, 64 of lo
constexpr uint32_t kWaitClocks = 400000000, kLookClocks = 20000;
constexpr float kMostSpan = 60.f;  // powers of two that a block's factors may reach over

struct LaChunkArgs {
    CUtensorMap x, y, z, out;  // [n_tok][heads][D], boxes of 128 tokens x 1 head x 64 columns
    LaRun run;
    float *states, *decays;  // [n_seq H][segments][D D]: the state before, then each segment's contribution but the last; [n_seq H][segments]
    int segments, per;       // per sequence; chunks of one
    int tma, tma_out, vec_out;  // tma: the maps are good (rows on 16 bytes); without, threads copy element by element
};

// Bytes of shared memory.
template <int D>
struct Smem {
    static constexpr int tile = L * D * 2;
    static constexpr int x = 0, sh = 5 * tile, sl = sh + D * D * 2;
    static constexpr int y(int i) { return i & 1 ? 2 * tile : tile; }
    static constexpr int z(int i) { return i & 1 ? 4 * tile : 3 * tile; }
    static constexpr int g = 6 * tile + (D == 128 ? tile : 0);  // five arrays of L floats (Gates), then barriers
    static constexpr int bars = g + 5 * L * 4, bytes = bars + 288;
    static_assert(sl + D * D * 2 <= g, "shared memory");
    // the first kernel: three stages of Y and Z
    static constexpr int stage(int i) { return i % 3 * 2 * tile; }
};
static_assert(Smem<128>::bytes <= kSmemPerCtaMax && Smem<64>::bytes <= kSmemPerCtaMax, "shared memory");

// mbarriers: products done, tiles loaded, buffers that may be loaded again (one arrival each; a barrier a buffer, since a load may be under
// way while the one before it has not arrived), then handovers (one arrival a warp).  A wait tells a phase from the one before it and the one
// behind it, no more: whoever waits for a phase has waited for the one before it, and the phase behind it comes only by way of
// something that this waiter does afterwards.
enum {
    kBarP, kBarXS, kBarS, kBarO, kLoadX, kLoadY, kLoadZ = kLoadY + 2, kFreeY = kLoadZ + 2, kFreeZ = kFreeY + 2, kSingle = kFreeZ + 2,
    kFullXY = kSingle, kFullZ, kFullS, kFullK, kFullP, kFreeO, kFullG, kFreeG, kFullW, kFreeW = kFullW + 2, kFullOut = kFreeW + 2, kBars = kFullOut + 2
};
// of the first kernel: products and stages read, stages loaded; of four chunks, Y' and gates made and the gates' sums so far
enum { kProduct = 0, kRead = kProduct + 2, kStage = kRead + 3, kMade = kStage + 3, kGates = kMade + 4, kCarry = kGates + 4, kTotal = kCarry + 4 };
static_assert((int)kTotal < (int)kBars, "barriers");

struct Gates {
    float *hi, *lo, *c;  // G in powers of two; e^(G of the block's last column - G)
    float* w;            // two buffers of cs e^(G_last - G)
    float* a;            // two of e^(G_last)
};

// What a CTA shares beside its tiles.
struct Shared {
    uint64_t* bars;
    float* decay;      // two
    long long* total;  // of a segment's gates, and whether a NaN was among them
    int* nan;
    uint32_t* tmem;
    volatile int* failed;
    uint64_t* drain;       // a barrier for what is in flight where a wait has given up
    volatile int* issued;  // loads (of the first kernel: of stages)
    __device__ __forceinline__ explicit Shared(char* at)
        : bars((uint64_t*)at), decay((float*)(at + 216)), total((long long*)(at + 224)), nan((int*)(at + 232)), tmem((uint32_t*)(at + 236)), failed((volatile int*)(at + 240)),
          drain((uint64_t*)(at + 248)), issued((volatile int*)(at + 256))
    {
        static_assert(kBars * 8 <= 216, "barriers");
    }
    // Until the barrier's phase is complete; gives up (false) after about 0.2 s (of SM clocks: reading the wall clock takes longer than most
    // waits here), and soon after another wait has given up: what follows then works on what it finds, which is nobody's
    // result, no more loads are issued, and the kernel ends (give_up()).
    __device__ __forceinline__ bool wait(int bar, uint32_t phase) const
    {
        const uint32_t a = tc::smem_addr(bars + bar);
        const uint32_t start = clock();
        for (;;) {
            uint32_t done;
            asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                         : "=r"(done)
                         : "r"(a), "r"(phase & 1)
                         : "memory");
            if (done) return true;
            const uint32_t now = (uint32_t)clock() - start;
            if (now > kLookClocks) {
                if (*failed) return false;
                if (now > kWaitClocks) {
                    *failed = 1;
                    return false;
                }
            }
        }
    }
    // One arrival of this warp, behind all its lanes.
    __device__ __forceinline__ void arrive(int bar) const
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bars + bar);
    }
};

// One lane of a whole warp, chosen so that the compiler knows that it is one: products issued by it take
// 68 cycles each, the tensor cores' own rate, where operands fetched from any one lane take up to 90.
__device__ __forceinline__ bool elect()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
// This warp's number, as a number of the whole warp.
__device__ __forceinline__ int warp_of(int tid) { return __shfl_sync(kFull, tid >> 5, 0); }

// 16 lanes x 16 columns: registers 2 i and 2 i + 1 are columns 4 i .. of lanes 0 .. 7 and 8 .. 15, thread = 4 lane + column.
__device__ __forceinline__ void st_16x128b(uint32_t at, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                 "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}

template <int ID, int T>
__device__ __forceinline__ void group_barrier()
{
    asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(T) : "memory");
}

// Two fp32 numbers as bf16 hi and lo words (the first in the low halves).
__device__ __forceinline__ void split2(f2 x, uint32_t& hi, uint32_t& lo)
{
    const float2 v = unpack2(x);
    hi = tc::pack_bf16x2(v.x, v.y);
    const float2 r = unpack2(add2(x, pack2(__uint_as_float((hi << 16) ^ 0x80000000u), __uint_as_float((hi & 0xffff0000u) ^ 0x80000000u))));
    lo = tc::pack_bf16x2(r.x, r.y);
}

// And what both leave out, exactly.
__device__ __forceinline__ uint32_t rest2(f2 x, uint32_t hi, uint32_t lo)
{
    const float2 v = unpack2(x);
    const float a = (v.x - __uint_as_float(hi << 16)) - __uint_as_float(lo << 16), b = (v.y - __uint_as_float(hi & 0xffff0000u)) - __uint_as_float(lo & 0xffff0000u);
    return tc::pack_bf16x2(a, b);
}

// A tile's rows in 128-byte swizzle: 64 columns a row, the next 64 columns 16 KB further.
__device__ __forceinline__ int swizzled(int row, int kc) { return (kc >> 3) * (L * 128) + row * 128 + (((kc & 7) ^ (row & 7)) << 4); }

__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int column, int head, int token, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(map), "r"(column), "r"(head), "r"(token), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map, int column, int head, int token)
{
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(map), "r"(column), "r"(head), "r"(token) : "memory");
}
// By one thread: 128 tokens from `token` on (rows outside the tensor read as zeros), whose bytes the barrier expects; and later ones into L2.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int head, long long token, uint64_t* bar)
{
#pragma unroll
    for (int c = 0; c < D; c += 64) tma_tile(dst + c * (L * 2), map, c, head, (int)token, tc::smem_addr(bar));
}
template <int D>
__device__ __forceinline__ void store_tile(const CUtensorMap* map, int head, long long token, uint32_t from)
{
#pragma unroll
    for (int c = 0; c < D; c += 64)
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(c), "r"(head), "r"((int)token),
                     "r"(from + c * (L * 2))
                     : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int D>
__device__ __forceinline__ void prefetch_tile(const CUtensorMap* map, int head, long long token)
{
    if (token < 0) return;
#pragma unroll
    for (int c = 0; c < D; c += 64) tma_prefetch(map, c, head, (int)token);
}

// The tile's rows [lo, hi) by T threads, element by element, and the others as zeros; or (copy false) the others alone.
template <int D, int T>
__device__ __forceinline__ void fill_tile(char* tile, const __nv_bfloat16* src, long long stride, long long token, int lo, int hi, bool copy, int tid)
{
#pragma unroll 1
    for (int u = tid; u < L * D / 8; u += T) {
        const int r = u / (D / 8), kc = u % (D / 8);
        const bool real = r >= lo && r < hi;
        if (real && !copy) continue;
        Pack<__nv_bfloat16, 8> p;
#pragma unroll
        for (int e = 0; e < 8; ++e) p.x[e] = real ? src[(token + r) * stride + 8 * kc + e] : __float2bfloat16(0.f);
        *reinterpret_cast<uint4*>(tile + swizzled(r, kc)) = *reinterpret_cast<const uint4*>(&p);
    }
}

// Log decays in fixed point: powers of two with 31 fraction bits.
constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.92596303e-8f;
__device__ __forceinline__ long long to_fixed(float gate)
{
    const float hi = gate * kLog2eHi, lo = fmaf(gate, kLog2eHi, -hi) + gate * kLog2eLo;
    const float whole = rintf(hi);
    return ((long long)__float2int_rn(whole) << 31) + (long long)__float2int_rn(((hi - whole) + lo) * 2147483648.f);
}
__device__ __forceinline__ float whole_of(long long x) { return (float)(int)(x >> 31); }
__device__ __forceinline__ float fraction_of(long long x) { return (float)(int)(x & 0x7fffffff) * 4.65661287e-10f; }
// The exponent of a sum, however long: 2^-1024 is 0 in fp32.
__device__ __forceinline__ float from_fixed(long long x)
{
    x = x < -(1ll << 41) ? -(1ll << 41) : x;
    return whole_of(x) + fraction_of(x);
}

// A lane's four gates of a chunk whose row 0 is the token `first`: those that enter before the walk's tokens 4 l .. 4 l + 3, for rows in [lo, hi)
// (0 elsewhere, and backwards behind the sequence's last token).  They are kept as stored until they are summed, so that loads are under way together.
struct RawGates {
    uint32_t v[4];
    __device__ __forceinline__ void load(const LaRun& A, const LaSequence& q, int h, long long first, int lo, int hi, int lane)
    {
        const char* p = (const char*)A.g;
        const long long at = (first + A.reverse) * A.gs0 + h * A.gs1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int pos = 4 * lane + k, r = A.reverse ? L - 1 - pos : pos;
            const bool real = r >= lo && r < hi && !(A.reverse && first + r + 1 >= q.hi);
            v[k] = 0;
            if (real) v[k] = A.gate_dtype == GDN_F32 ? ((const uint32_t*)p)[at + r * A.gs0] : ((const uint16_t*)p)[at + r * A.gs0];
        }
    }
    __device__ __forceinline__ float get(int k, int dtype) const
    {
        float g = __uint_as_float(v[k]);
        if (dtype == GDN_BF16) g = __uint_as_float(v[k] << 16);
        if (dtype == GDN_F16) g = __half2float(__ushort_as_half((unsigned short)v[k]));
        return g < kLaLeastGate ? kLaLeastGate : g > kLaMostGate ? kLaMostGate : g;
    }
};

// The running sums of a chunk's 128 gates by one warp: lane l has the walk's tokens 4 l .. 4 l + 3.
struct GateSums {
    long long at[4], end, all;  // after each token, after the lane's block of 32, after all
    uint32_t nan;               // bit k: a NaN up to token k; bit 4: in the block; bit 5: anywhere
    __device__ __forceinline__ GateSums(const RawGates& raw, int dtype, int lane)
    {
        float gate[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) gate[k] = raw.get(k, dtype);
        bool bad = false;
        nan = 0;
        long long x = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            bad |= gate[k] != gate[k];
            nan |= (bad ? 1u : 0u) << k;
            x += gate[k] == gate[k] ? to_fixed(gate[k]) : 0;
            at[k] = x;
        }
        const long long own = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(kFull, x, o);
            if (lane >= o) x += y;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) at[k] += x - own;
        all = __shfl_sync(kFull, x, 31);
        end = __shfl_sync(kFull, x, lane | 7);
        const uint32_t lanes = __ballot_sync(kFull, bad);
        if (lanes & ((1u << lane) - 1)) nan |= 15;
        if (lanes >> (lane & 24) & 255) nan |= 16;
        if (lanes) nan |= 32;
    }
};
// Four numbers of a lane, in walking order, to an array in the rows' order.
__device__ __forceinline__ void put4(float* array, bool reverse, int lane, const float (&v)[4])
{
    *reinterpret_cast<float4*>(array + (reverse ? L - 4 - 4 * lane : 4 * lane)) = reverse ? make_float4(v[3], v[2], v[1], v[0]) : make_float4(v[0], v[1], v[2], v[3]);
}

// Y'^T = (w Y)^T as bf16 hi and lo into TMEM, by PARTS x 4 warps: a warp's 32 lanes of TMEM are columns of Y, and it takes 128 / PARTS
// tokens.  A transposing load of 8 tokens x 8 columns leaves a lane two tokens of one column, which is where TMEM's 16 x 128-bit shape wants them.  With THIRD, the rest goes to
// `third`.
template <int D, int PARTS, bool THIRD>
__device__ __forceinline__ void decayed_keys(uint32_t tile, uint32_t tmem, uint32_t third, const float* w, int quarter, int part, int lane)
{
    if (32 * quarter < D) {
#pragma unroll 1
        for (int t0 = part * (L / PARTS); t0 < (part + 1) * (L / PARTS); t0 += 32) {
            f2 ww[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) ww[b] = *reinterpret_cast<const f2*>(w + t0 + 8 * b + 2 * (lane & 3));
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                uint32_t hi[8], lo[8], rest[8];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t at = tile + swizzled(t0 + lane, 4 * quarter + 2 * h + c);
                    uint32_t v[4];
                    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                                 : "r"(at)
                                 : "memory");
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const f2 x = mul2(pack2(__uint_as_float(v[b] << 16), __uint_as_float(v[b] & 0xffff0000u)), ww[b]);
                        split2(x, hi[2 * b + c], lo[2 * b + c]);
                        if (THIRD) rest[2 * b + c] = rest2(x, hi[2 * b + c], lo[2 * b + c]);
                    }
                }
                const uint32_t lanes = ((uint32_t)(32 * quarter + 16 * h) << 16) + t0 / 2;
                st_16x128b(tmem + lanes, hi);
                st_16x128b(tmem + lanes + 64, lo);
                if (THIRD) st_16x128b(third + lanes, rest);
            }
        }
        tc::wait_st();
    }
}

// Operands in shared memory.  Of tiles in 128-byte swizzle: K-major (tokens are M or N; 32 bytes a slice of 16 columns, 16 KB every 64)
// and MN-major (columns are N; 16 rows a slice).  Of S^T, rows i, in core matrices of 8 x 8: MN-major.
constexpr uint64_t kSwizzle128 = 2ull << 61;
__device__ __forceinline__ uint64_t swizzled_k(uint32_t tile) { return tc::make_desc(tile, 16, 1024) | kSwizzle128; }
__device__ __forceinline__ uint64_t swizzled_mn(uint32_t tile) { return tc::make_desc(tile, L * 128, 1024) | kSwizzle128; }
__device__ __forceinline__ uint64_t step_k(int s) { return (uint64_t)((s >> 2) * (L * 128) + (s & 3) * 32) >> 4; }
__device__ __forceinline__ uint64_t step_mn(int s) { return (uint64_t)(s * 2048) >> 4; }
constexpr uint32_t kTransposedB = 1u << 16;

// dS^T (+)= Y'^T Z.  M is 128 for D = 64 too: lanes 64 .. 127 are nobody's.
template <int D, bool THIRD>
__device__ __forceinline__ void issue_state(uint32_t to, uint32_t y, uint32_t third, uint32_t z, bool accumulate)
{
    constexpr uint32_t idesc = tc::idesc_bf16(D) | kTransposedB;
    const uint64_t b = swizzled_mn(z);
#pragma unroll 4
    for (int s = 0; s < L / 16; ++s) {
        tc::mma_ts16(to, y + 8 * s, b + step_mn(s), idesc, accumulate || s > 0);
        tc::mma_ts16(to, y + 64 + 8 * s, b + step_mn(s), idesc, 1);
        if (THIRD) tc::mma_ts16(to, third + 8 * s, b + step_mn(s), idesc, 1);
    }
}
template <int D>
__device__ __forceinline__ void issue_scores(uint32_t tmem, uint32_t x, uint32_t y)
{
    const uint64_t a = swizzled_k(x), b = swizzled_k(y);
#pragma unroll
    for (int s = 0; s < D / 16; ++s) tc::mma_ss16(tmem + kColP, a + step_k(s), b + step_k(s), tc::idesc_bf16(L), s > 0);
}
template <int D>
__device__ __forceinline__ void issue_state_output(uint32_t tmem, uint32_t x, uint32_t sh, uint32_t sl)
{
    constexpr uint32_t idesc = tc::idesc_bf16(D) | kTransposedB;
    const uint64_t a = swizzled_k(x), bh = tc::make_desc(sh, D * 16, 128), bl = tc::make_desc(sl, D * 16, 128);
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        tc::mma_ss16(tmem + kColO, a + step_k(s), bh + s * D * 2, idesc, s > 0);
        tc::mma_ss16(tmem + kColO, a + step_k(s), bl + s * D * 2, idesc, 1);
    }
}
// Of every 32 columns of P, 16 hold hi words and 16 lo words.
template <int D>
__device__ __forceinline__ void issue_output(uint32_t tmem, uint32_t z)
{
    constexpr uint32_t idesc = tc::idesc_bf16(D) | kTransposedB;
    const uint64_t b = swizzled_mn(z);
#pragma unroll 4
    for (int s = 0; s < L / 16; ++s) {
        const uint32_t a = tmem + kColP + 32 * (s >> 1) + 8 * (s & 1);
        tc::mma_ts16(tmem + kColO, a, b + step_mn(s), idesc, 1);
        tc::mma_ts16(tmem + kColO, a + 16, b + step_mn(s), idesc, 1);
    }
}

// What both kernels begin with: barriers (arrivals(i) of barrier i) and tensor memory.
template <typename F>
__device__ __forceinline__ uint32_t begin(const Shared& sh, F&& arrivals)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i) tc::mbar_init(sh.bars + i, arrivals(i));
        tc::mbar_init(sh.drain, 1);
        *sh.issued = 0;
        tc::mbar_fence_init();
        *sh.failed = 0;
    }
    if (threadIdx.x < 32) tc::tmem_alloc(sh.tmem, kTmemCols);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    return *sh.tmem;
}

// The last `buffers` of n loads that took turns at barriers from `bar` on.
__device__ __forceinline__ bool landed(const Shared& sh, int bar, int buffers, int n)
{
    bool done = true;
    for (int i = n > buffers ? n - buffers : 0; i < n; ++i) done &= tc::mbar_wait(sh.bars + bar + i % buffers, (i / buffers) & 1);
    return done;
}
// Where a wait has given up, products and loads may still be in flight, whose tensor and shared memory are another CTA's once this one is gone: waits for them, each for
// 0.2 s at most.  Out of line, so that the code that always runs stays short (inlined: a prompt of 32768 tokens 174 us, so 173).
__device__ __noinline__ void give_up(char* shared, bool segments)
{
    const Shared sh(shared);
    const int warp = warp_of(threadIdx.x), n = *sh.issued;
    if (threadIdx.x == 0) atomicOr(&g_la_chunk_status[1], 1);
    bool done = true;
    if (warp == kIssuer && elect()) {
        tc::commit(sh.drain);
        done = tc::mbar_wait(sh.drain, 0);
    } else if (warp == kLoader && elect()) {
        if (segments) done = landed(sh, kStage, 3, n);
        else  // in the order Y, X, Z
            done = landed(sh, kLoadY, 2, (n + 2) / 3) & landed(sh, kLoadX, 1, (n + 1) / 3) & landed(sh, kLoadZ, 2, n / 3);
    }
    if (!done) atomicOr(&g_la_chunk_status[1], 2);
    __syncthreads();
}
// What both kernels end with.
__device__ __forceinline__ void end(const Shared& sh, uint32_t tmem, int warp, bool segments)
{
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (*sh.failed) give_up((char*)sh.bars, segments);
    if (warp == 0) tc::tmem_free(tmem, kTmemCols);
}

__device__ __forceinline__ float* state_of(const LaChunkArgs& A, int D, int nh, int segment)
{
    return A.states + ((long long)nh * A.segments + segment) * D * D;
}

// Columns j in [c0, c0 + N) of row i of S^T; in memory rows follow each other in S^T's order (`rows`) or in S's.
template <int D, int N>
__device__ __forceinline__ void load_state(float (&m)[N], const float* head, int i, int c0, bool rows)
{
    if (rows) {
#pragma unroll
        for (int c = 0; c < N; c += 4) {
            const float4 v = *reinterpret_cast<const float4*>(head + i * D + c0 + c);
            m[c] = v.x;
            m[c + 1] = v.y;
            m[c + 2] = v.z;
            m[c + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; ++c) m[c] = head[(c0 + c) * D + i];
    }
}
template <int D, int N>
__device__ __forceinline__ void store_state(const float (&m)[N], float* head, int i, int c0, bool rows)
{
    if (rows) {
#pragma unroll
        for (int c = 0; c < N; c += 4) *reinterpret_cast<float4*>(head + i * D + c0 + c) = make_float4(m[c], m[c + 1], m[c + 2], m[c + 3]);
    } else {
#pragma unroll
        for (int c = 0; c < N; ++c) head[(c0 + c) * D + i] = m[c];
    }
}

// The chunks [c0, c1) of segment `segment` of a sequence, in walking order; last: no segment follows.
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

// What a CTA works on.
struct Work {
    LaSequence q;
    Part part;
    uint32_t tmem;
    int h, nh, segment, count;
    bool reverse;
    // Of the segment's chunk i: the token of its row 0, and its real rows [lo, hi).  Backwards, chunks are cut from
    // the sequence's end, rows stay in the tokens' order.
    __device__ __forceinline__ long long token(int i) const
    {
        const long long at = (part.c0 + i) * L;
        return reverse ? q.hi - L - at : q.lo + at;
    }
    __device__ __forceinline__ int lo(int i) const
    {
        const long long t = token(i);
        return t < q.lo ? (int)(q.lo - t) : 0;
    }
    __device__ __forceinline__ int hi(int i) const
    {
        const long long left = q.hi - token(i);
        return left < L ? (int)left : L;
    }
    __device__ __forceinline__ bool whole(int i) const { return lo(i) == 0 && hi(i) == L; }
    // Whether threads write its tiles: without TMA, and where rows are another sequence's (of TMA's, one chunk of a segment at most).
    __device__ __forceinline__ bool made(const LaChunkArgs& A, int i) const { return !A.tma || !whole(i); }
};

__device__ __forceinline__ const __nv_bfloat16* head_of(const void* p, int h, int heads, long long stride)
{
    return (const __nv_bfloat16*)p + (h % heads) * stride;
}

// Segment contributions: segments - 1 CTAs a sequence and head.  With THIRD, for the token form by segments, to fp32: what its dq and dk are off by adds up in dg.
template <int D, bool THIRD>
__global__ void __launch_bounds__(kThreads, 1) la_segment_kernel(const __grid_constant__ LaChunkArgs A)
{
    using S = Smem<D>;
    extern __shared__ __align__(1024) char sm[];
    const Shared sh(sm + S::bars);
    float* sw = reinterpret_cast<float*>(sm + S::g);
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_of(tid);
    const int per_seq = A.segments - 1;
    Work W;
    W.nh = blockIdx.x / per_seq;
    W.segment = blockIdx.x - W.nh * per_seq;
    const int n = W.nh / A.run.H;
    W.h = W.nh - n * A.run.H;
    W.reverse = A.run.reverse;
    begin_after();
    W.q = la_sequence(A.run, n);
    if (!W.q.ok) return;  // the second kernel reports it
    W.part = part_of(A, W.q.hi - W.q.lo, W.segment);
    if (W.part.none || W.part.last) return;
    const uint32_t tmem = begin(sh, [&](int i) { return i >= kMade && i < kGates ? 16 : i >= kGates && i < kCarry ? 1 + A.run.held : 1; }), base = tc::smem_addr(sm);
    const int count = (int)(W.part.c1 - W.part.c0), yh = W.h % A.run.yh, zh = W.h % A.run.zh;
    // whole chunks, from the last one back: the sequence's last one is the last segment's
    auto token = [&](int it) { return W.token(count - 1 - it); };
    // two buffers of Y' and of its weights, three stages of Y and Z
    auto keys = [&](int it) { return tmem + kColY - 128 * (it & 1); };
    auto third = [&](int it) { return tmem + kColO + 64 * (it & 1); };
    if (warp == kLoader) {
        if (A.tma && elect()) {
            int it = 0;
            for (; it < count; ++it) {
                if (it >= 3 && !sh.wait(kRead + it % 3, it / 3 - 1)) break;
                uint64_t* bar = sh.bars + kStage + it % 3;
                tc::mbar_expect_tx(bar, 2 * S::tile);
                load_tile<D>(base + S::stage(it), &A.y, yh, token(it), bar);
                load_tile<D>(base + S::stage(it) + S::tile, &A.z, zh, token(it), bar);
                if (it + 2 < count) {
                    prefetch_tile<D>(&A.y, yh, token(it + 2));
                    prefetch_tile<D>(&A.z, zh, token(it + 2));
                }
            }
            *sh.issued = it;
        }
        __syncwarp();
    } else if (warp == kIssuer) {
        for (int it = 0; it < count; ++it) {
            if (A.tma) sh.wait(kStage + it % 3, it / 3);
            sh.wait(kMade + (it & 3), it >> 2);
            tc::fence_after();
            if (elect()) {
                issue_state<D, THIRD>(tmem, keys(it), third(it), base + S::stage(it) + S::tile, it > 0);
                tc::commit(sh.bars + kProduct + (it & 1));
                tc::commit(sh.bars + kRead + it % 3);
            }
            __syncwarp();
        }
    } else if (warp >= kWriters && warp < kWriters + 4) {
        // the gates: a warp sums every fourth chunk, and gets the sum of those behind it from the warp before
        long long* sums = reinterpret_cast<long long*>(sw + 4 * L);
        int* nans = reinterpret_cast<int*>(sums + 4);
        RawGates next;
        auto gates = [&](int it) {
            if (it < count) next.load(A.run, W.q, W.h, token(it), 0, L, lane);
        };
        gates(warp - kWriters);
        for (int it = warp - kWriters; it < count; it += 4) {
            const GateSums s(next, A.run.gate_dtype, lane);
            gates(it + 4);
            long long carry = 0;
            bool nan = false;  // among the gates behind
            if (it > 0) {
                sh.wait(kCarry + ((it - 1) & 3), (it - 1) >> 2);
                carry = sums[(it - 1) & 3];
                nan = nans[(it - 1) & 3] != 0;
            }
            nan |= (s.nan & 32) != 0;
            if (lane == 0) {
                sums[it & 3] = carry + s.all;
                nans[it & 3] = nan;
            }
            sh.arrive(kCarry + (it & 3));
            float w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = nan ? NAN : ex2(from_fixed(carry + (s.all - s.at[k])));
            if (it > 3) sh.wait(kMade + (it & 3), (it >> 2) - 1);  // the weights before these have been read
            put4(sw + L * (it & 3), W.reverse, lane, w);
            sh.arrive(kGates + (it & 3));
            if (it == count - 1) {
                if (lane == 0) {
                    *sh.total = carry + s.all;
                    *sh.nan = nan;
                }
                sh.arrive(kTotal);
            }
        }
    } else if (warp < 16) {
        for (int it = 0; it < count; ++it) {
            const float* w = sw + L * (it & 3);
            if (it > 1) sh.wait(kProduct + (it & 1), (it >> 1) - 1);  // the product before the last has read Y', which all warps had made
            if (A.tma) sh.wait(kStage + it % 3, it / 3);
            else {
                if (it > 2) sh.wait(kRead + it % 3, it / 3 - 1);
                fill_tile<D, 512>(sm + S::stage(it), head_of(A.run.y, W.h, A.run.yh, A.run.ys1), A.run.ys0, token(it), 0, L, true, tid);
                fill_tile<D, 512>(sm + S::stage(it) + S::tile, head_of(A.run.z, W.h, A.run.zh, A.run.zs1), A.run.zs0, token(it), 0, L, true, tid);
                tc::fence_async_smem();
                group_barrier<2, 512>();
            }
            sh.wait(kGates + (it & 3), it >> 2);
            tc::fence_after();
            decayed_keys<D, 4, THIRD>(base + S::stage(it), keys(it), third(it), w, warp & 3, warp >> 2, lane);
            tc::fence_before();
            sh.arrive(kMade + (it & 3));
        }
        if (count > 1) sh.wait(kProduct + (count & 1), (count - 2) >> 1);
        sh.wait(kProduct + ((count - 1) & 1), (count - 1) >> 1);
        sh.wait(kTotal, 0);
        const long long carry = *sh.total;
        const bool nan = *sh.nan != 0;
        tc::fence_after();
        constexpr int C = D / 4;  // columns of a thread
        const int row = 32 * (warp & 3) + lane, c0 = (warp >> 2) * C;
        float d[C];
        if constexpr (C == 32) tc::ld32(tc::taddr(tmem, warp, 0) + c0, d);
        else tc::ld16(tc::taddr(tmem, warp, 0) + c0, d);
        tc::wait_ld();
        if (row < D && !*sh.failed) {
            const float all = nan ? NAN : ex2(from_fixed(carry));
#pragma unroll
            for (int i = 0; i < C; ++i) d[i] *= A.run.cs;
            if (W.segment == 0) {
                // the state before it, kept for the segment's own start too (the last segment may replace it in place)
                float m[C];
#pragma unroll
                for (int i = 0; i < C; ++i) m[i] = 0.f;
                if (W.q.in >= 0) load_state<D>(m, A.run.s_in + W.q.in * A.run.in_stride + (long long)W.h * D * D, row, c0, A.run.transposed_in);
                store_state<D>(m, state_of(A, D, W.nh, 0), row, c0, true);
#pragma unroll
                for (int i = 0; i < C; ++i) d[i] = fmaf(all, m[i], d[i]);
            }
            store_state<D>(d, state_of(A, D, W.nh, W.segment + 1), row, c0, true);
            if (tid == 0) A.decays[W.nh * A.segments + W.segment + 1] = all;
        }
    }
    end(sh, tmem, warp, true);
}

// 32 consecutive bytes.
__device__ __forceinline__ void st_global32(void* p, const uint32_t (&v)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
                 "r"(v[6]), "r"(v[7])
                 : "memory");
}

// The first group: P', and the state's part of the output scaled.
template <int D>
__device__ __forceinline__ void scores(const LaChunkArgs& A, const Work& W, const Shared& sh, const Gates& g)
{
    constexpr int H = D / 2;  // columns of a thread's output
    const int tid = threadIdx.x, lane = tid & 31, warp = warp_of(tid), quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;
    const uint32_t lanes = tc::taddr(W.tmem, warp, 0);

    for (int i = 0; i < W.count; ++i) {
        sh.wait(kFullG, i);
        const float gh = g.hi[row], gl = g.lo[row], eg = ex2(gh + gl);
        sh.wait(kBarP, i);
        tc::fence_after();
        // P' in the place of P: every 32 columns become 16 of hi words and 16 of lo words
#pragma unroll 1
        for (int b = 2 * half; b < 2 * half + 2; ++b) {
            uint32_t ph[16], pl[16];
            if (W.reverse ? b < quarter : b > quarter) {
#pragma unroll
                for (int e = 0; e < 16; ++e) ph[e] = pl[e] = 0u;
            } else {
                float p[32];
                tc::ld32(lanes + kColP + 32 * b, p);
                const int last = W.reverse ? 32 * b : 32 * b + 31, first = W.reverse ? 32 * b + 31 : 32 * b;
                // columns that the walk has met: all of them, or of the diagonal block those of the lanes below and this one (backwards, above)
                const uint32_t met = b != quarter ? 0xffffffffu : W.reverse ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);
                // a factor of the row and one of the column, where both are far from fp32's limits
                if (b != quarter || fabsf(g.hi[first] - g.hi[last]) < kMostSpan) {
                    const float rf = ex2((gh - g.hi[last]) + (gl - g.lo[last])) * A.run.cs;
                    const f2 rr = pack2(rf, rf);
                    tc::wait_ld();
                    if (b == quarter) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) p[e] = met >> e & 1 ? p[e] : 0.f;
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(g.c + 32 * b + e);
                        split2(mul2(pack2(p[e], p[e + 1]), mul2(rr, c.x)), ph[e / 2], pl[e / 2]);
                        split2(mul2(pack2(p[e + 2], p[e + 3]), mul2(rr, c.y)), ph[e / 2 + 1], pl[e / 2 + 1]);
                    }
                } else {
                    tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 uh = *reinterpret_cast<const float2*>(g.hi + 32 * b + e), ul = *reinterpret_cast<const float2*>(g.lo + 32 * b + e);
                        const float x0 = met >> e & 1 ? p[e] * (ex2((gh - uh.x) + (gl - ul.x)) * A.run.cs) : 0.f;
                        const float x1 = met >> (e + 1) & 1 ? p[e + 1] * (ex2((gh - uh.y) + (gl - ul.y)) * A.run.cs) : 0.f;
                        split2(pack2(x0, x1), ph[e / 2], pl[e / 2]);
                    }
                }
            }
            tc::st16(lanes + kColP + 32 * b, ph);
            tc::st16(lanes + kColP + 32 * b + 16, pl);
        }
        sh.arrive(kFreeG);
        // e^G X S^T
        sh.wait(kBarXS, i);
        tc::fence_after();
#pragma unroll 1
        for (int c = 0; c < H; c += 32) {
            float o[32];
            uint32_t u[32];
            tc::ld32(lanes + kColO + half * H + c, o);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * eg);
            tc::st32(lanes + kColO + half * H + c, u);
        }
        tc::wait_st();
        tc::fence_before();
        sh.arrive(kFullP);
    }
}

// The third group: the output, a row a thread.
template <int D>
__device__ __forceinline__ void writes(const LaChunkArgs& A, const Work& W, char* sm, const Shared& sh)
{
    using S = Smem<D>;
    const int lane = threadIdx.x & 31, warp = warp_of(threadIdx.x) - kWriters, row = 32 * warp + lane;
    const uint32_t lanes = tc::taddr(W.tmem, warp, kColO);
    for (int i = 0; i < W.count; ++i) {
        // a whole chunk through Z's buffer, which is free until the second chunk behind this one
        const bool staged = A.tma_out && W.whole(i), real = row >= W.lo(i) && row < W.hi(i);
        const long long at = ((W.token(i) + row) * A.run.H + W.h) * D;
        sh.wait(kBarO, i);
        tc::fence_after();
        if (staged || (A.vec_out && A.run.out_dtype == GDN_BF16)) {
            // all columns first, so that the next chunk's product may have their place
            uint32_t v[D / 2];
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tc::ld32(lanes + c, o);
                tc::wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) v[c / 2 + k] = tc::pack_bf16x2(A.run.co * o[2 * k], A.run.co * o[2 * k + 1]);
            }
            tc::fence_before();
            sh.arrive(kFreeO);
            if (staged) {
#pragma unroll
                for (int k = 0; k < D / 8; ++k)
                    *reinterpret_cast<uint4*>(sm + S::z(i) + swizzled(row, k)) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            } else if (real) {
#pragma unroll
                for (int k = 0; k < D / 8; ++k)
                    *reinterpret_cast<uint4*>((__nv_bfloat16*)A.run.out + at + 8 * k) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
            __syncwarp();
        } else {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tc::ld32(lanes + c, o);
                tc::wait_ld();
                if (c + 32 == D) {
                    tc::fence_before();
                    sh.arrive(kFreeO);
                }
                if (real && A.vec_out && A.run.out_dtype == GDN_F32) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(A.run.co * o[e + k]);
                        st_global32((float*)A.run.out + at + c + e, v);
                    }
                } else if (real) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) st_any(A.run.out, at + c + e, A.run.out_dtype, A.run.co * o[e]);
                }
                __syncwarp();
            }
        }
        if (staged) tc::fence_async_smem();
        sh.arrive(kFullOut + (i & 1));
    }
}

// The second group: Y' and the state (of y's and dv's runs, whose states lie as the pool's do).
template <int D>
__device__ __forceinline__ void states(const LaChunkArgs& A, const Work& W, char* sm, const Shared& sh, const Gates& g)
{
    using S = Smem<D>;
    constexpr int H = D / 2;  // columns of a thread's state row
    const int tid = threadIdx.x - kGroup, lane = tid & 31, warp = warp_of(tid), quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;
    const uint32_t base = tc::smem_addr(sm), lanes = tc::taddr(W.tmem, warp, 0);
    const bool has_state = row < D;

    // the state before the segment
#pragma unroll 1
    for (int c = half * H; c < half * H + H; c += 16) {
        float m[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) m[e] = 0.f;
        if (has_state) {
            if (W.segment > 0) {
#pragma unroll 1
                for (int s = 1; s <= W.segment; ++s) {
                    float d[16];
                    load_state<D>(d, state_of(A, D, W.nh, s), row, c, true);
                    const float a = s > 1 ? A.decays[W.nh * A.segments + s] : 0.f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) m[e] = s > 1 ? fmaf(a, m[e], d[e]) : d[e];
                }
            } else if (!W.part.last) {
                load_state<D>(m, state_of(A, D, W.nh, 0), row, c, true);
            } else if (W.q.in >= 0) {
                load_state<D>(m, A.run.s_in + W.q.in * A.run.in_stride + (long long)W.h * D * D, row, c, false);
            }
        }
        uint32_t u[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(m[e]);
        tc::st16(lanes + kColS + c, u);
    }
    tc::wait_st();

    for (int i = 0; i < W.count; ++i) {
        const bool made = W.made(A, i);
        const int lo = W.lo(i), hi = W.hi(i);
        if (A.tma) sh.wait(kLoadY + (i & 1), i >> 1);
        if (made) {  // rows of Y and Z that are another sequence's become zeros: theirs may hold anything
            if (!A.tma && i > 0) sh.wait(kBarXS, i - 1);
            if (!A.tma) fill_tile<D, kGroup>(sm + S::x, head_of(A.run.x, W.h, A.run.xh, A.run.xs1), A.run.xs0, W.token(i), lo, hi, true, tid);
            fill_tile<D, kGroup>(sm + S::y(i), head_of(A.run.y, W.h, A.run.yh, A.run.ys1), A.run.ys0, W.token(i), lo, hi, !A.tma, tid);
            tc::fence_async_smem();
            group_barrier<2, kGroup>();
            sh.arrive(kFullXY);
        }
        sh.wait(kFullW + (i & 1), i >> 1);
        const float a = g.a[i & 1];
        const f2 aa = pack2(a, a);
        // S as it enters the chunk, for X S^T; a S, for dS to be added to
        if (A.tma && i > 0) sh.wait(kBarXS, i - 1);
        if (32 * quarter < D) {
#pragma unroll 1
            for (int c = half * H; c < half * H + H; c += 16) {
                float m[16];
                uint32_t u[16];
                tc::ld16(lanes + kColS + c, m);
                tc::wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    uint4 h, l;
                    split2(pack2(m[e], m[e + 1]), h.x, l.x);
                    split2(pack2(m[e + 2], m[e + 3]), h.y, l.y);
                    split2(pack2(m[e + 4], m[e + 5]), h.z, l.z);
                    split2(pack2(m[e + 6], m[e + 7]), h.w, l.w);
                    const int at = ((row >> 3) * (D / 8) + (c + e) / 8) * 128 + (row & 7) * 16;
                    *reinterpret_cast<uint4*>(sm + S::sh + at) = h;
                    *reinterpret_cast<uint4*>(sm + S::sl + at) = l;
                }
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 v = unpack2(mul2(pack2(m[e], m[e + 1]), aa));
                    u[e] = __float_as_uint(v.x);
                    u[e + 1] = __float_as_uint(v.y);
                }
                tc::st16(lanes + kColS + c, u);
            }
            tc::fence_async_smem();
        }
        sh.arrive(kFullS);
        decayed_keys<D, 2, false>(base + S::y(i), W.tmem + kColY, 0, g.w + L * (i & 1), quarter, half, lane);
        tc::wait_st();
        tc::fence_before();
        sh.arrive(kFullK);
        sh.arrive(kFreeW + (i & 1));
        if (made) {
            if (A.tma) sh.wait(kLoadZ + (i & 1), i >> 1);
            else if (i > 0) sh.wait(kBarO, i - 1);
            fill_tile<D, kGroup>(sm + S::z(i), head_of(A.run.z, W.h, A.run.zh, A.run.zs1), A.run.zs0, W.token(i), lo, hi, !A.tma, tid);
            tc::fence_async_smem();
            sh.arrive(kFullZ);
        }
        sh.wait(kBarS, i);
        tc::fence_after();
    }
    if (has_state && W.part.last && W.q.out >= 0 && !__any_sync(kFull, *sh.failed)) {
        float a = 1.f;  // backwards, the state before the first token
        if (W.reverse && W.q.hi > W.q.lo) a = expf(ld_any(A.run.g, W.q.lo * A.run.gs0 + W.h * A.run.gs1, A.run.gate_dtype));
        float* to = A.run.s_out + W.q.out * A.run.out_stride + (long long)W.h * D * D;
#pragma unroll 1
        for (int c = half * H; c < half * H + H; c += 16) {
            float m[16];
            tc::ld16(lanes + kColS + c, m);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) m[e] *= a;
            store_state<D>(m, to, row, c, false);
        }
    }
}

// The thread that issues all products of the segment, in order.
template <int D>
__device__ __forceinline__ void products(const LaChunkArgs& A, const Work& W, uint32_t base, const Shared& sh)
{
    using S = Smem<D>;
    for (int i = 0; i < W.count; ++i) {
        const bool made = W.made(A, i);
        if (A.tma) {
            sh.wait(kLoadX, i);
            sh.wait(kLoadY + (i & 1), i >> 1);
        }
        if (made) sh.wait(kFullXY, A.tma ? 0 : i);
        if (i > 0) sh.wait(kBarO, i - 1);  // P' has been read
        tc::fence_after();
        issue_scores<D>(W.tmem, base + S::x, base + S::y(i));
        tc::commit(sh.bars + kBarP);
        sh.wait(kFullS, i);
        if (i > 0) sh.wait(kFreeO, i - 1);
        tc::fence_after();
        issue_state_output<D>(W.tmem, base + S::x, base + S::sh, base + S::sl);
        tc::commit(sh.bars + kBarXS);
        if (A.tma) sh.wait(kLoadZ + (i & 1), i >> 1);
        if (made) sh.wait(kFullZ, A.tma ? 0 : i);
        sh.wait(kFullK, i);
        tc::fence_after();
        issue_state<D, false>(W.tmem + kColS, W.tmem + kColY, 0, base + S::z(i), true);
        tc::commit(sh.bars + kBarS);
        tc::commit(sh.bars + kFreeY + (i & 1));
        sh.wait(kFullP, i);
        tc::fence_after();
        issue_output<D>(W.tmem, base + S::z(i));
        tc::commit(sh.bars + kBarO);
    }
}

// The thread that stores whole chunks, and frees Z's buffers.
template <int D>
__device__ __forceinline__ void stores(const LaChunkArgs& A, const Work& W, uint32_t base, const Shared& sh)
{
    for (int i = 0; i < W.count; ++i) {
        sh.wait(kFullOut + (i & 1), i >> 1);
        if (A.tma_out && W.whole(i)) {
            store_tile<D>(&A.out, W.h, W.token(i), base + Smem<D>::z(i));
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        tc::mbar_arrive(sh.bars + kFreeZ + (i & 1));
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// The warp that sums the gates.
__device__ __forceinline__ void sum_gates(const LaChunkArgs& A, const Work& W, const Shared& sh, const Gates& g)
{
    const int lane = threadIdx.x & 31;
    RawGates next[2];  // of this chunk and the one behind it
    auto gates = [&](RawGates& to, int i) {
        if (i < W.count) to.load(A.run, W.q, W.h, W.token(i), W.lo(i), W.hi(i), lane);
    };
    gates(next[0], 0);
    gates(next[1], 1);
    for (int i = 0; i < W.count; ++i) {
        const GateSums s(next[0], A.run.gate_dtype, lane);
        next[0] = next[1];
        gates(next[1], i + 2);
        float hi[4], lo[4], w[4], c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            hi[k] = s.nan >> k & 1 ? NAN : whole_of(s.at[k]);
            lo[k] = fraction_of(s.at[k]);
            w[k] = s.nan & 32 ? NAN : A.run.cs * ex2(from_fixed(s.all - s.at[k]));
            c[k] = s.nan & 16 ? NAN : ex2(from_fixed(s.end - s.at[k]));
        }
        if (i > 1) sh.wait(kFreeW + (i & 1), (i >> 1) - 1);
        put4(g.w + L * (i & 1), W.reverse, lane, w);
        if (lane == 0) g.a[i & 1] = s.nan & 32 ? NAN : ex2(from_fixed(s.all));
        sh.arrive(kFullW + (i & 1));
        if (i > 0) sh.wait(kFreeG, i - 1);
        put4(g.hi, W.reverse, lane, hi);
        put4(g.lo, W.reverse, lane, lo);
        put4(g.c, W.reverse, lane, c);
        sh.arrive(kFullG);
    }
}

// The thread that issues all loads.
template <int D>
__device__ __forceinline__ void loads(const LaChunkArgs& A, const Work& W, uint32_t base, const Shared& sh)
{
    using S = Smem<D>;
    const int xh = W.h % A.run.xh, yh = W.h % A.run.yh, zh = W.h % A.run.zh;
    auto load = [&](uint32_t to, const CUtensorMap* map, int head, int i, int bar) {
        tc::mbar_expect_tx(sh.bars + bar, S::tile);
        load_tile<D>(to, map, head, W.token(i), sh.bars + bar);
    };
    auto issued = [&](int n) { *sh.issued = n; };
    for (int i = 0; i < W.count; ++i) {
        if (i > 1 && !sh.wait(kFreeY + (i & 1), (i >> 1) - 1)) return issued(3 * i);
        load(base + S::y(i), &A.y, yh, i, kLoadY + (i & 1));
        if (i > 0 && !sh.wait(kBarXS, i - 1)) return issued(3 * i + 1);
        load(base + S::x, &A.x, xh, i, kLoadX);
        if (i > 1 && !sh.wait(kFreeZ + (i & 1), (i >> 1) - 1)) return issued(3 * i + 2);
        load(base + S::z(i), &A.z, zh, i, kLoadZ + (i & 1));
    }
    issued(3 * W.count);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) la_chunk_kernel(const __grid_constant__ LaChunkArgs A)
{
    using S = Smem<D>;
    extern __shared__ __align__(1024) char sm[];
    const Shared sh(sm + S::bars);
    float* g0 = reinterpret_cast<float*>(sm + S::g);
    const Gates g = {g0, g0 + L, g0 + 2 * L, g0 + 3 * L, sh.decay};
    Work W;
    W.nh = blockIdx.x / A.segments;
    W.segment = blockIdx.x - W.nh * A.segments;
    const int n = W.nh / A.run.H;
    W.h = W.nh - n * A.run.H;
    W.reverse = A.run.reverse;
    begin_after();
    W.q = la_sequence(A.run, n);
    if (!W.q.ok) {
        if (threadIdx.x == 0) atomicOr(&g_la_chunk_status[0], 1);
        return;
    }
    W.part = part_of(A, W.q.hi - W.q.lo, W.segment);
    if (W.part.none) return;
    W.count = W.part.c1 > W.part.c0 ? (int)(W.part.c1 - W.part.c0) : 0;
    W.tmem = begin(sh, [&](int i) { return i < kSingle ? 1 : i == kFullG || i == kFullW || i == kFullW + 1 ? 1 + A.run.held : i == kFreeO || i >= kFullOut ? 4 : 8; });
    const int warp = warp_of(threadIdx.x);
    const uint32_t base = tc::smem_addr(sm);
    if (warp < 8) scores<D>(A, W, sh, g);
    else if (warp < kWriters) states<D>(A, W, sm, sh, g);
    else if (warp < kIssuer) writes<D>(A, W, sm, sh);
    else if (warp == kSummer) sum_gates(A, W, sh, g);
    else if (warp == kIssuer && elect()) products<D>(A, W, base, sh);
    else if (warp == kLoader && A.tma && elect()) loads<D>(A, W, base, sh);
    else if (warp == kStorer && elect()) stores<D>(A, W, base, sh);
    end(sh, W.tmem, warp, false);
}

// Segments a sequence and head, s of p chunks each: at most as many as leave every SM one, and those of the least p + s, since
// a segment more costs about what a chunk more does (the states that the last one starts from).  Against one segment of c chunks, 3 us a chunk,
// the first kernel costs a launch and 1.6 times the rest: 8 heads of 128, a prompt of 1024 tokens 36 us in one segment and 36 in 3, of 2048
// 60 and 47, of 4096 106 and 56 (6 segments; 70 with 16), of 16384 388 and 98 (12); 32 heads, 2048 tokens 60 us and 52 (4), 512 tokens 25 and
// 36; 64 heads, 2048 tokens 62 and 64 (2), 4096 tokens 109 and 98.
void plan(const LaRun& A, int* segments, int* per)
{
    const long long heads = (long long)A.n_seq * A.H;
    const long long chunks = ((long long)A.T + L - 1) / L;
    long long most = heads > 0 ? kNumSMs / heads : 1;
    if (most > kMostSegments) most = kMostSegments;
    *segments = 1;
    *per = (int)chunks;
    long long best = (5 * chunks - 5) / 8;
    for (long long s = 2; s <= most && s <= chunks; ++s) {
        const long long p = (chunks + s - 1) / s, real = (chunks + p - 1) / p;
        if (p + real >= best) continue;
        best = p + real;
        *segments = (int)real;
        *per = (int)p;
    }
}

// A map of [n_tok][heads][D]: false where its rows do not lie on 16 bytes, or are otherwise nothing for TMA.
bool make_map(CUtensorMap* map, const void* ptr, long long s0, long long s1, int heads, int n_tok, int D)
{
    typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                               const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r);
        return e == cudaSuccess && r == cudaDriverEntryPointSuccess ? (Encode)f : (Encode) nullptr;
    }();
    if (heads == 1) s1 = D;
    if (n_tok == 1) s0 = (long long)heads * D;
    if (!encode || n_tok < 1 || (uintptr_t)ptr % 16 || s0 % 8 || s1 % 8 || s0 < 1 || s1 < 1 || s0 >= (1ll << 38) || s1 >= (1ll << 38)) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)n_tok}, strides[2] = {(cuuint64_t)s1 * 2, (cuuint64_t)s0 * 2};
    const cuuint32_t box[3] = {64, 1, L}, ones[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What the segments leave, but the last.
template <int D, bool THIRD>
int launch_segments(const LaChunkArgs& A, cudaStream_t st)
{
    if (A.segments < 2) return 0;
    const int e = (int)cudaFuncSetAttribute(la_segment_kernel<D, THIRD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::bytes);
    return e ? e : launch_after(la_segment_kernel<D, THIRD>, (unsigned)(A.run.n_seq * A.run.H * (A.segments - 1)), kThreads, Smem<D>::bytes, st, A);
}
template <int D>
int launch(const LaChunkArgs& A, cudaStream_t st)
{
    int e = (int)cudaFuncSetAttribute(la_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::bytes);
    if (!e) e = launch_segments<D, false>(A, st);
    if (!e) e = launch_after(la_chunk_kernel<D>, (unsigned)(A.run.n_seq * A.run.H * A.segments), kThreads, Smem<D>::bytes, st, A);
    return e;
}

}  // namespace

// From 32 tokens on, a chunk's fixed cost is less than that many steps: 32 heads of 128, 31 tokens 23 us token by token and 17 in a chunk (24 tokens 19
// and 17), 2048 heads 203 and 177 (24 tokens 162 and 177).  Of many heads of 64, half as wide a step, only from 48 on: 1024 heads, 40 tokens 60 us and
// 60, 48 tokens 70 and 60, 768 heads, 32 tokens 48 and 50; 384 heads, 32 tokens 29 and 29, 40 tokens 33 and 29; 256 heads, 32 tokens 27 and 21; 32 heads, 21 and 13.
bool la_chunk_fits(const la_params_t* p)
{
    const int least = p->S_k == 64 && p->n_seq * p->H_v > 4 * kNumSMs ? 48 : 32;
    return p->in_dtype == GDN_BF16 && p->S_k == p->S_v && (p->S_k == 64 || p->S_k == 128) && p->T >= least;
}

size_t la_chunk_workspace(const LaRun& A)
{
    int segments, per;
    plan(A, &segments, &per);
    return segments > 1 ? (size_t)A.n_seq * A.H * segments * ((size_t)A.DK * A.DV + 1) * sizeof(float) : 0;
}

static LaChunkArgs args_of(const LaRun& run, void* workspace, int segments, int per)
{
    LaChunkArgs A{};
    A.run = run;
    A.segments = segments;
    A.per = per;
    A.states = (float*)workspace;
    A.decays = A.states + (long long)run.n_seq * run.H * A.segments * run.DK * run.DV;
    A.tma = make_map(&A.x, run.x, run.xs0, run.xs1, run.xh, run.n_tok, run.DK) && make_map(&A.y, run.y, run.ys0, run.ys1, run.yh, run.n_tok, run.DK) &&
            make_map(&A.z, run.z, run.zs0, run.zs1, run.zh, run.n_tok, run.DV);
    A.tma_out = A.tma && run.out_dtype == GDN_BF16 && make_map(&A.out, run.out, (long long)run.H * run.DV, run.DV, run.H, run.n_tok, run.DV);
    A.vec_out = (uintptr_t)run.out % 32 == 0;
    return A;
}

int launch_la_chunk(const LaRun& run, void* workspace, cudaStream_t st)
{
    int segments, per;
    plan(run, &segments, &per);
    const LaChunkArgs A = args_of(run, workspace, segments, per);
    return run.DK == 128 ? launch<128>(A, st) : launch<64>(A, st);
}

// Segments for the token form: as many as fill the places that its CTAs of 64 rows have, of whole chunks, but eight at most, each of which reads what those before
// it left.  48 heads of 128, gradients of 4096 tokens: one segment 5012 us, 6 segments 1701; nine sequences of up to 500 tokens, 8 heads of 64: 429 and (4) 247.  More than
// eight would be faster for few heads: 4 heads of 64, 4096 tokens, 16 segments 305 us and 32 250 against 468, 6 heads of 128 702 and 572 against 669; dg stays as exact.
static void plan_tokens(const LaRun& A, int* segments, int* per)
{
    const long long ctas = (long long)A.n_seq * A.H * (A.DV / 64), chunks = ((long long)A.T + L - 1) / L;
    long long s = ctas > 0 ? 4 * kNumSMs / ctas : 1;
    if (s > 8) s = 8;
    if (s > chunks) s = chunks;
    if (s < 1) s = 1;
    *per = (int)((chunks + s - 1) / s);
    *segments = *per > 0 ? (int)((chunks + *per - 1) / *per) : 1;
}

size_t la_tokens_workspace(const LaRun& A)
{
    int segments, per;
    plan_tokens(A, &segments, &per);
    return segments > 1 ? (size_t)A.n_seq * A.H * segments * ((size_t)A.DK * A.DV + 1) * sizeof(float) : 0;
}

int launch_la_tokens(const LaRun& run, int dtype, void* workspace, cudaStream_t st)
{
    LaRun B = run;
    int segments, per;
    plan_tokens(run, &segments, &per);
    if (segments > 1) {
        const LaChunkArgs A = args_of(run, workspace, segments, per);
        const int e = run.DK == 128 ? launch_segments<128, true>(A, st) : launch_segments<64, true>(A, st);
        if (e) return e;
        B.segments = segments;
        B.per = per * L;
        B.states = A.states;
        B.decays = A.decays;
    }
    return launch_la_token(B, dtype, st);
}

int la_chunk_take_status(void* stream, bool bad_too, int* timeout, int* bad)
{
    int words[2] = {0, 0};
    int e = la_read_words(g_la_chunk_status, stream, 2, words);
    *timeout = words[1];
    if (!e && words[1]) e = la_clear_word(g_la_chunk_status, stream, 1);
    else if (!e && words[0] && bad_too) {
        *bad = words[0];
        e = la_clear_word(g_la_chunk_status, stream, 0);
    }
    return e;
}

}  // namespace gdn
