// distill_rows.cu -- distillation from a teacher's top logits (include/distill.h) where a row fits a CTA.
//
// CTAs that walk rows, each with a row in registers and the next one
// on its way to shared memory by asynchronous copies, every thread's packs to places of its own, so that nothing but the row's reductions
// (maximum, then sum) needs a barrier.  The list is a thread's business each: index and teacher's logit arrive a row ahead, and its softmax takes the same
// two reductions.
//
// Bytes bound it, the row in and the gradient out: 8192 bf16 rows of 32000, loss and gradient 201 us (78 % of the copy rate; issue slots 56 %, two
// exponentials an element), the gradient alone 161 us (98 %; 28 more where lse is far from zero and the rows are summed again); 4096 fp32 rows of 32000, one CTA an SM, 177 us (89 %) and
// 165 (96 %).
#include "distill_internal.h"
#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_rows.cuh"

namespace gdn {
namespace {

constexpr int kRowThreads = 256, kWideThreads = 512, kRowMostPacks = 16;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) { asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory"); }

// A maximum over a warp as whole numbers of the same order; NaN does not count.
__device__ __forceinline__ float warp_max(float x)
{
    const unsigned b = __float_as_uint(x + 0.f), o = x != x ? 0u : b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
    const unsigned m = __reduce_max_sync(kFull, o);
    return m == 0u ? -INFINITY : __uint_as_float(m ^ ((unsigned)((int)~m >> 31) | 0x80000000u));
}
__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}

// Two neighbours, rounded together.
__device__ __forceinline__ void put2(float* y, float a, float b)
{
    y[0] = a;
    y[1] = b;
}
__device__ __forceinline__ void put2(__nv_bfloat16* y, float a, float b) { *reinterpret_cast<uint32_t*>(y) = tc::pack_bf16x2(a, b); }
__device__ __forceinline__ void put2(__half* y, float a, float b) { *reinterpret_cast<__half2*>(y) = __floats2half2_rn(a, b); }

// CTAs an SM, by the registers that a row's packs take.
constexpr int rows_resident(int threads, int packs) { return threads == kWideThreads ? 1 : packs == 16 ? 2 : packs == 8 ? 3 : 4; }

template <typename T, int THREADS, int PACKS, int MODE>
__global__ void __launch_bounds__(THREADS, rows_resident(THREADS, PACKS)) distill_rows_kernel(const DistillArgs A, int rows)
{
    constexpr int VEC = 16 / (int)sizeof(T), WARPS = THREADS / 32;
    extern __shared__ __align__(16) char ring[];  // PACKS x THREADS packs: the next row's
    __shared__ __align__(16) int s_idx[THREADS];
    __shared__ __align__(16) float s_p[THREADS];
    __shared__ float s_max[2][WARPS], s_sum[2][WARPS], s_loss[WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t place = tc::smem_addr(ring) + 16 * tid;  // + 16 THREADS p
    begin_after();

    auto row_of = [&](long long r) { return segment_of((const T*)A.logits + r * A.row_stride, 0, A.seg, A.V); };
    auto fetch = [&](long long r) {
        if (r < rows) {
            const Segment<T> s = row_of(r);
#pragma unroll
            for (int p = 0; p < PACKS; ++p) {
                const int at = (p * THREADS + tid) * VEC;
                if (at >= s.lo && at + VEC <= s.end) cp_async16(place + p * (16 * THREADS), s.at + at);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // The gradient alone of large fp32 rows reads lse again, from L2, behind the next row's copies: its stores then come after them and not between, 16384 rows of 8000 164 us
    // instead of 178, 4096 of 32000 164 instead of 176 (608 of them 35 instead of 32; smaller rows 101 instead of 93, 16-bit ones 177 instead of 167).
    constexpr bool again = MODE == kGradient && sizeof(T) == 4 && PACKS >= 8;
    int next_idx = -1;
    float next_t = -INFINITY, next_lse = 0.f;
    auto list = [&](long long r) {
        next_idx = -1;
        if (tid < A.K && r < rows) {
            next_idx = A.indices[r * A.K + tid];
            next_t = ld_any(A.teacher, r * A.K + tid, A.teacher_dtype);
        }
        if (MODE == kGradient && r < rows) next_lse = __ldcg(A.lse_in + r);
    };
    fetch(blockIdx.x);
    list(blockIdx.x);
    for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
        const Segment<T> s = row_of(r);
        const T* in = (const T*)A.logits + r * A.row_stride;
        // the list: this row's entry of the thread, and the student's logit of it
        const bool entry = next_idx >= 0 && next_idx < A.V && next_t != -INFINITY;
        const int idx = entry ? next_idx : -1;
        const float t = entry ? next_t : -INFINITY;
        float xj = 0.f;
        if (entry) xj = to_f32(in[idx]);
        const float dloss = MODE == kLoss ? 0.f : A.dloss[r], lse = next_lse;
        list(r + gridDim.x);
        const bool sums = MODE != kGradient || fabsf(lse) > kMostLse;
        // the row, from where its copies have landed; its first and last elements where 16 bytes cut them
        Pack<T, VEC> x[PACKS];
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        {
            Pack<T, VEC> none;
#pragma unroll
            for (int i = 0; i < VEC; ++i) none.x[i] = from_f32<T>(-INFINITY);
            unsigned cut = 0;
#pragma unroll
            for (int p = 0; p < PACKS; ++p) {
                const int at = (p * THREADS + tid) * VEC;
                const bool whole = at >= s.lo && at + VEC <= s.end;
                x[p] = none;
                if (whole) x[p] = *reinterpret_cast<const Pack<T, VEC>*>(ring + 16 * (tid + p * THREADS));
                cut |= (at < s.end && !whole ? 1u : 0u) << p;
            }
            while (cut) {
                const int c = __ffs(cut) - 1, at = (c * THREADS + tid) * VEC;
                cut &= cut - 1;
                Pack<T, VEC> part = none;
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (at + i >= s.lo && at + i < s.end) part.x[i] = s.at[at + i];
#pragma unroll
                for (int p = 0; p < PACKS; ++p)
                    if (p == c) x[p] = part;
            }
        }
        float m = -INFINITY;
        if (sums) {
#pragma unroll
            for (int p = 0; p < PACKS; ++p) m = fmaxf(m, pack_max(x[p]));
            m = warp_max(m);
        }
        const float tm = warp_max(t);
        if (lane == 0) {
            s_max[0][warp] = m;
            s_max[1][warp] = tm;
        }
        const bool any = __syncthreads_or(entry);  // the last row's list and gradients are done with too
        fetch(r + gridDim.x);
        m = warp_max(s_max[0][lane & (WARPS - 1)]);
        const float top = warp_max(s_max[1][lane & (WARPS - 1)]);
        const float tj = (t - top) * A.inv_tau, ej = entry ? expf(tj) : 0.f;
        // q = 2^((x - base) L - off)
        float sum = 0.f, base = 0.f, off = 0.f;
        if (sums) {
            base = base_of(m);
            const f2 ll = pack2(A.L, A.L), bb = pack2(-base, -base);
            f2 s2 = 0;
#pragma unroll
            for (int p = 0; p < PACKS; ++p)
#pragma unroll
                for (int i = 0; i < VEC; i += 2) {
                    const float2 v = unpack2(mul2(add2(x[p].pair(i), bb), ll));
                    s2 = add2(s2, pack2(ex2(v.x), ex2(v.y)));
                }
            sum = warp_sum(sum2(s2));
        }
        const float es = warp_sum(ej);
        if (lane == 0) {
            s_sum[0][warp] = sum;
            s_sum[1][warp] = es;
        }
        s_idx[tid] = idx;
        __syncthreads();
        sum = s_sum[0][lane & (WARPS - 1)];
        float esum = s_sum[1][lane & (WARPS - 1)];
#pragma unroll
        for (int o = WARPS / 2; o >= 1; o >>= 1) {
            sum += __shfl_xor_sync(kFull, sum, o);
            esum += __shfl_xor_sync(kFull, esum, o);
        }
        const float pj = ej / esum;
        if (MODE != kGradient) {
            const float log_s = logf(sum);
            if (warp * 32 < A.K || warp == 0) {
                float l = 0.f;
                // p first: a masked token's distance over tau may leave fp32's range where p of it does not
                if (entry && pj != 0.f) l = xj == -INFINITY && sum == sum ? INFINITY : pj * ((tj - logf(esum)) + log_s) - pj * (xj - m) * A.inv_tau;
                l = warp_sum(l);
                if (lane == 0) s_loss[warp] = l;
            }
            if (tid == 0) A.lse[r] = !any ? 0.f : m == -INFINITY && sum == 0.f ? -INFINITY : fmaf(m, A.inv_tau, log_s);
        }
        if (sums) off = m == -INFINITY && sum == 0.f ? 0.f : log2f(sum);  // nothing but -inf: 2^-inf is 0
        else off = (again ? __ldcg(A.lse_in + r) : lse) * kLog2e;
        const float scale = dloss * A.inv_tau;
        if (MODE != kLoss) {
            // kept as stored: what the sum made of them would take twice the registers
            if (MODE != kLoss) {
#pragma unroll
                for (int p = 0; p < PACKS; ++p) {
                    uint4& w = reinterpret_cast<uint4&>(x[p]);
                    asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w));
                }
            }
            // scale q, the scale's magnitude in the exponent
            T* out = (T*)A.dlogits + r * A.d_stride;
            T* to = out + (s.at - in);
            const bool alike = (((uintptr_t)out ^ (uintptr_t)in) & 15) == 0;
            const float shift = off - log2f(fabsf(scale));
            const uint32_t sign = scale < 0.f ? (sizeof(T) == 2 ? 0x80008000u : 0x80000000u) : 0u, keep = any ? 0xffffffffu : 0u;
            const f2 ll = pack2(A.L, A.L), rr = pack2(-shift, -shift), bb = pack2(-base, -base);
#pragma unroll
            for (int p = 0; p < PACKS; ++p) {
                const int at = (p * THREADS + tid) * VEC;
                Pack<T, VEC> y;
#pragma unroll
                for (int i = 0; i < VEC; i += 2) {
                    const float2 v = unpack2(fma2(add2(x[p].pair(i), bb), ll, rr));
                    put2(y.x + i, ex2(v.x), ex2(v.y));
                }
                uint4& w = *reinterpret_cast<uint4*>(&y);
                w = make_uint4((w.x ^ sign) & keep, (w.y ^ sign) & keep, (w.z ^ sign) & keep, (w.w ^ sign) & keep);
                if (alike && at >= s.lo && at + VEC <= s.end) *reinterpret_cast<uint4*>(to + at) = w;
                else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (at + i >= s.lo && at + i < s.end) to[at + i] = y.x[i];
                }
            }
        }
        s_p[tid] = pj;
        __syncthreads();
        if (MODE != kGradient && tid == 0) {
            float l = 0.f;
            for (int w = 0; w < WARPS && (w == 0 || w * 32 < A.K); ++w) l += s_loss[w];
            A.loss[r] = any ? l : 0.f;
        }
        if (MODE != kLoss && entry) {
            float p = 0.f;  // of every entry of this token
            for (int e = 0; e < A.K; e += 4) {
                const int4 i4 = *reinterpret_cast<const int4*>(s_idx + e);
                if (i4.x == idx || i4.y == idx || i4.z == idx || i4.w == idx) {
                    const float4 p4 = *reinterpret_cast<const float4*>(s_p + e);
                    p += (i4.x == idx ? p4.x : 0.f) + (i4.y == idx ? p4.y : 0.f) + (i4.z == idx ? p4.z : 0.f) + (i4.w == idx ? p4.w : 0.f);
                }
            }
            ((T*)A.dlogits + r * A.d_stride)[idx] = from_f32<T>(scale * (ex2(fmaf(xj - base, A.L, -off)) - p));
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T, int THREADS, int PACKS, int MODE>
int launch_rows(DistillArgs A, int64_t N, cudaStream_t st)
{
    constexpr int bytes = PACKS * THREADS * 16;
    A.seg = PACKS * THREADS * (16 / (int)sizeof(T));
    if (bytes > 40 * 1024) {
        const int e = (int)cudaFuncSetAttribute(distill_rows_kernel<T, THREADS, PACKS, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e) return e;
    }
    const int64_t most = rows_resident(THREADS, PACKS) * kNumSMs;
    return launch_after(distill_rows_kernel<T, THREADS, PACKS, MODE>, (unsigned)(N < most ? N : most), THREADS, bytes, st, A, (int)N);
}
template <typename T, int MODE>
int launch_rows(const distill_params_t* p, const DistillArgs& A, cudaStream_t st)
{
    const int vec = 16 / (int)sizeof(T);
    const int64_t packs = (p->V + 2 * vec - 2) / vec;
    return packs <= 4 * kRowThreads    ? launch_rows<T, kRowThreads, 4, MODE>(A, p->N, st)
           : packs <= 8 * kRowThreads  ? launch_rows<T, kRowThreads, 8, MODE>(A, p->N, st)
           : packs <= 16 * kRowThreads ? launch_rows<T, kRowThreads, 16, MODE>(A, p->N, st)
                                       : launch_rows<T, kWideThreads, 16, MODE>(A, p->N, st);
}

template <int MODE>
int launch_mode(const distill_params_t* p, const DistillArgs& A, cudaStream_t st)
{
    return p->dtype == GDN_F32    ? launch_rows<float, MODE>(p, A, st)
           : p->dtype == GDN_BF16 ? launch_rows<__nv_bfloat16, MODE>(p, A, st)
                                  : launch_rows<__half, MODE>(p, A, st);
}

constexpr int kLeastWide = kNumSMs / 2;

}  // namespace

// Rows that a CTA of the rows' kernel walks: up to 64 KB, or of many rows 128 KB, with a list of no more entries than it has threads.  Loss and gradient of
// bf16 rows of 32000, against clusters (with the call's 6 us of an idle GPU): 1 row 11 us and 11, 64 rows 11 and 13, 200 rows 15 and 21, 1216 rows 39 and 48,
// 4096 rows 107 and 147; rows of 8000: 1 row 9 and 11, 200 rows 9 and 13, 4096 rows 42 and 57.  fp32 rows of 32000, one CTA an SM: 1 row 11 and 11, 64 rows 14
// and 15 (the gradient alone 13 and 13), 100 rows 13 and 21, 300 rows 21 and 29, 4096 rows 177 and 291.
bool distill_walks_rows(const distill_params_t* p)
{
    const int vec = 16 / (int)elem_size(p->dtype);
    const int64_t packs = (p->V + 2 * vec - 2) / vec;
    return p->K <= kRowThreads && p->V >= vec && (packs <= kRowThreads * kRowMostPacks || (packs <= kWideThreads * kRowMostPacks && p->N >= kLeastWide));
}

int launch_distill_rows(const distill_params_t* p, const DistillArgs& A, int mode, cudaStream_t st)
{
    return mode == kLoss ? launch_mode<kLoss>(p, A, st) : mode == kBoth ? launch_mode<kBoth>(p, A, st) : launch_mode<kGradient>(p, A, st);
}

}  // namespace gdn
