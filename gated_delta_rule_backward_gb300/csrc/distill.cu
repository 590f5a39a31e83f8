// distill.cu -- distillation from a teacher's top logits: loss, gradient, or both from one reading of the
// logits (include/distill.h).
//
// Rows of up to 64 KB, and many of up to 128 KB, are walked by CTAs (distill_rows.cu).
//
// Any other row belongs to a cluster of 1 to 8 CTAs, each of which holds its part in registers (up to 8 packs of 16 bytes for
// each of up to 512 threads: 512 KB a row in all), so that the maximum, the sum of exponentials and the gradient come
// from one reading; longer rows are walked in chunks and read again for the gradient.  Every thread sums
// against its own maximum, and (maximum, sum) pairs are joined in fixed order: over the warp, the CTA, and the cluster,
// whose CTAs write theirs into each other's shared memory before one cluster barrier.  The list is the first warp's work, while the row's loads are in
// flight: p_j, log p_j, and the student's logits of the listed tokens, read before any gradient may replace them.
//
// With L = log2(e) / tau, exp((x - m) / tau) = 2^((x - m) L).  The gradient is written dense, q alone; the few
// listed tokens are written again behind a barrier, from the numbers kept, so that each is rounded once.
//
// Bytes bound it, the row in and the gradient out, but 50 % of the copy rate is what it reaches with loss and gradient, 62 with the gradient alone and 40 with the loss (2048 bf16
// rows of 128257: 317, 255 and 197 us; of 151936, which fill 58 % of eight CTAs' registers, 606, 425 and 377; 2048 fp32 rows of 50001 277, 220 and 178): a
// CTA's registers hold one row, and nothing is under way while it is summed.  For a few rows latency does.
#include <cfloat>
#include <cmath>
#include <cstdio>

#include "distill_internal.h"
#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "gdn_launch.cuh"
#include "gdn_rows.cuh"

namespace gdn {
namespace {

constexpr int kMostK = 1024, kMostThreads = 512, kMostPacks = 8, kMostCtas = 8;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Writes a pair into the shared memory of the cluster's CTA `rank`, at the place that `here` has in this CTA.
__device__ __forceinline__ void st_cluster(float2* here, uint32_t rank, float2 v)
{
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_addr(here)), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(v.x), "f"(v.y) : "memory");
}

// (a maximum, the sum of 2^((x - maximum) L) against it); (-inf, 0) where there is nothing.
__device__ __forceinline__ float2 join(float2 a, float2 b, float L)
{
    const float m = fmaxf(a.x, b.x);
    const float s = (a.x == m ? a.y : a.y * ex2((a.x - m) * L)) + (b.x == m ? b.y : b.y * ex2((b.x - m) * L));
    return make_float2(m, s);
}

template <typename T, int VEC, int PACKS>
__device__ __forceinline__ float2 max_and_sum(const Pack<T, VEC> (&x)[PACKS], float L)
{
    float m = -INFINITY;
#pragma unroll
    for (int p = 0; p < PACKS; ++p) m = fmaxf(m, pack_max(x[p]));
    const float base = base_of(m);
    const f2 bb = pack2(-base, -base), ll = pack2(L, L);
    f2 s2 = 0;
#pragma unroll
    for (int p = 0; p < PACKS; ++p)
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            const float2 v = unpack2(mul2(add2(x[p].pair(i), bb), ll));
            s2 = add2(s2, pack2(ex2(v.x), ex2(v.y)));
        }
    return make_float2(m, sum2(s2));
}

template <typename T, int PACKS, int MODE>
__global__ void __launch_bounds__(kMostThreads, 2) distill_kernel(const DistillArgs A)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    __shared__ int s_idx[kMostK];                                // -1: no entry
    __shared__ float s_p[kMostK], s_x[kMostK], s_log[kMostK];
    __shared__ float2 s_warp[kMostThreads / 32], s_cta[kMostCtas];
    __shared__ int s_any;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
    const long long row = blockIdx.x / A.ctas;
    const int rank = blockIdx.x - (int)(row * A.ctas);           // clusters are consecutive CTAs
    const T* in = (const T*)A.logits + row * A.row_stride;
    const long long lead = (long long)(((uintptr_t)in & 15) / sizeof(T));
    const long long lo = (long long)rank * A.chunks * A.seg - lead, hi = lo + (long long)A.chunks * A.seg;  // this CTA's columns
    if (MODE != kGradient && A.ctas > 1) cluster_arrive();  // the others have started before their shared memory is written
    begin_after();

    auto load = [&](Pack<T, VEC>(&x)[PACKS], int c) {
        ld_chunk_packs<T, VEC, PACKS>(x, segment_of(in, rank * A.chunks + c, A.seg, A.V), [&](int p) { return (p * threads + tid) * VEC; });
    };
    // Whether the row has an entry is known to the first warp alone, so the first chunk is on its way before.
    Pack<T, VEC> x[PACKS];
    const float lse = MODE == kGradient ? A.lse_in[row] : 0.f;
    load(x, 0);
    if (warp == 0) {
        const int* idx = A.indices + row * A.K;
        bool any = false;
        float top = -INFINITY;
        for (int j = lane; j < A.K; j += 32) {
            const int i = idx[j];
            const float t = ld_any(A.teacher, row * A.K + j, A.teacher_dtype);
            const bool entry = i >= 0 && i < A.V && t != -INFINITY;
            any |= entry;
            s_idx[j] = entry ? i : -1;
            s_log[j] = entry ? t : -INFINITY;
            // the gradient alone looks at its own columns only: the others' may already hold gradients
            s_x[j] = entry && (MODE != kGradient || (i >= lo && i < hi)) ? to_f32(in[i]) : 0.f;
            if (entry) top = fmaxf(top, t);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        float sum = 0.f;
        for (int j = lane; j < A.K; j += 32) {
            const float t = (s_log[j] - top) * A.inv_tau, e = s_idx[j] >= 0 ? expf(t) : 0.f;
            s_log[j] = t;
            s_p[j] = e;
            sum += e;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        const float inv = 1.f / sum, log_sum = logf(sum);
        for (int j = lane; j < A.K; j += 32)
            if (s_idx[j] >= 0) {
                s_p[j] *= inv;
                s_log[j] -= log_sum;
            }
        any = __any_sync(kFull, any);
        if (lane == 0) s_any = any;
    }

    float base = 0.f, off = 0.f;
    if (MODE != kGradient || fabsf(lse) > kMostLse) {
        float2 ms = max_and_sum<T, VEC, PACKS>(x, A.L);
        for (int c = 1; c < A.chunks; ++c) {
            load(x, c);
            ms = join(ms, max_and_sum<T, VEC, PACKS>(x, A.L), A.L);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) ms = join(ms, make_float2(__shfl_xor_sync(kFull, ms.x, o), __shfl_xor_sync(kFull, ms.y, o)), A.L);
        if (lane == 0) s_warp[warp] = ms;
        __syncthreads();
        if (warp == 0) {
            ms = lane < threads / 32 ? s_warp[lane] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) ms = join(ms, make_float2(__shfl_xor_sync(kFull, ms.x, o), __shfl_xor_sync(kFull, ms.y, o)), A.L);
        }
        if (A.ctas > 1) {
            if (MODE == kGradient) cluster_arrive();
            cluster_wait();
            if (warp == 0 && lane < A.ctas) st_cluster(&s_cta[rank], lane, ms);
            cluster_arrive();
            cluster_wait();
        } else {
            if (tid == 0) s_cta[0] = ms;
            __syncthreads();
        }
        ms = s_cta[0];
        for (int i = 1; i < A.ctas; ++i) ms = join(ms, s_cta[i], A.L);
        if (MODE != kGradient && rank == 0 && warp == 0) {
            const bool nothing = ms.x == -INFINITY && ms.y == 0.f;  // every logit is -inf
            const float log_s = logf(ms.y);
            float l = 0.f;
            for (int j = lane; j < A.K; j += 32)
                if (s_idx[j] >= 0 && s_p[j] != 0.f) {
                    const float xj = s_x[j];
                    // p first: a masked token's distance over tau may leave fp32's range where p of it does not
                    l += xj == -INFINITY && ms.y == ms.y ? INFINITY : s_p[j] * (s_log[j] + log_s) - s_p[j] * (xj - ms.x) * A.inv_tau;
                }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
            if (lane == 0) {
                A.loss[row] = s_any ? l : 0.f;
                A.lse[row] = !s_any ? 0.f : nothing ? -INFINITY : fmaf(ms.x, A.inv_tau, log_s);
            }
        }
        if (MODE == kLoss) return;
        // q = 2^((x - base) L - off), base the largest logit: one number for both would be off by half an ulp of m L powers of two
        off = ms.x == -INFINITY && ms.y == 0.f ? 0.f : log2f(ms.y);  // every logit is -inf: q = 0
        base = base_of(ms.x);
    } else {
        __syncthreads();
        off = lse * kLog2e;
    }

    // the gradient: scale q, then the listed tokens again
    const bool any = s_any;
    const float scale = any ? A.dloss[row] * A.inv_tau : 0.f;
    T* out = (T*)A.dlogits + row * A.d_stride;
    const bool alike = (((uintptr_t)out ^ (uintptr_t)in) & 15) == 0;
    const f2 ll = pack2(A.L, A.L), rr = pack2(-off, -off), bb = pack2(-base, -base);
    for (int c = 0; c < A.chunks; ++c) {
        if (A.chunks > 1) load(x, c);
        const Segment<T> s = segment_of(in, rank * A.chunks + c, A.seg, A.V);
        T* to = out + (s.at - in);
#pragma unroll
        for (int p = 0; p < PACKS; ++p) {
            const int at = (p * threads + tid) * VEC;
            Pack<T, VEC> y;
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                const float2 v = unpack2(fma2(add2(x[p].pair(i), bb), ll, rr));
                y.x[i] = from_f32<T>(any ? scale * ex2(v.x) : 0.f);
                y.x[i + 1] = from_f32<T>(any ? scale * ex2(v.y) : 0.f);
            }
            if (alike && at >= s.lo && at + VEC <= s.end) *reinterpret_cast<uint4*>(to + at) = *reinterpret_cast<const uint4*>(&y);
            else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (at + i >= s.lo && at + i < s.end) to[at + i] = y.x[i];
            }
        }
    }
    if (!any) return;
    __syncthreads();
    for (int j = tid; j < A.K; j += threads) {
        const int i = s_idx[j];
        if (i < 0 || i < lo || i >= hi) continue;
        float p = 0.f;  // of every entry of this token
        for (int e = 0; e < A.K; ++e) p += s_idx[e] == i ? s_p[e] : 0.f;
        out[i] = from_f32<T>(scale * (ex2(fmaf(s_x[j] - base, A.L, -off)) - p));
    }
}

int fail(int s, const char* msg)
{
    set_last_error(msg);
    return s;
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

int check(const distill_params_t* p)
{
    if (!p) return fail(GDN_ERR_INVALID_ARG, "distill: params is NULL");
    if (p->N < 0 || p->K < 0 || p->V < 1) return fail(GDN_ERR_INVALID_ARG, "distill: N and K must be >= 0, V >= 1");
    if (p->row_stride < p->V || p->d_stride < p->V) return fail(GDN_ERR_INVALID_ARG, "distill: a row stride is below V");
    if (!known_dtype(p->dtype) || !known_dtype(p->teacher_dtype)) return fail(GDN_ERR_INVALID_ARG, "distill: unknown dtype");
    // below the smallest normal number log2(e) / tau is infinite, and a distance of 0 times it NaN
    if (!(p->temperature >= FLT_MIN) || std::isinf(p->temperature))
        return fail(GDN_ERR_INVALID_ARG, "distill: the temperature must be finite and at least the smallest normal number");
    if (p->K > kMostK) return fail(GDN_ERR_UNSUPPORTED, "distill: more than 1024 entries a row");
    if (p->V > (1 << 30) || p->N > (1 << 30) / kMostCtas) return fail(GDN_ERR_UNSUPPORTED, "distill: V or N is too large");
    return GDN_OK;
}

// How a row is laid over CTAs: as few as hold it in registers, and more where that would leave SMs without one.
struct Plan {
    int ctas, threads, packs, chunks, seg;
};
Plan plan_of(const distill_params_t* p)
{
    const int vec = 16 / (int)elem_size(p->dtype);
    const int64_t packs = (p->V + 2 * vec - 2) / vec;  // the row may start vec - 1 elements into its first
    Plan pl{1, 128, 2, 1, 0};
    while (pl.ctas < kMostCtas && (packs > (int64_t)pl.ctas * kMostThreads * kMostPacks || (p->N * pl.ctas < 2 * kNumSMs && packs > pl.ctas * 512))) pl.ctas *= 2;
    while (pl.threads < kMostThreads && packs > (int64_t)pl.ctas * pl.threads * 4) pl.threads *= 2;
    while (pl.packs < kMostPacks && packs > (int64_t)pl.ctas * pl.threads * pl.packs) pl.packs *= 2;
    const int64_t most = (int64_t)pl.threads * pl.packs;
    pl.chunks = (int)((packs + pl.ctas * most - 1) / (pl.ctas * most));
    const int64_t parts = (int64_t)pl.ctas * pl.chunks;
    pl.seg = (int)((packs + parts - 1) / parts) * vec;
    return pl;
}

template <typename T, int MODE>
int launch(DistillArgs A, const Plan& pl, int64_t N, cudaStream_t st)
{
    A.seg = pl.seg;
    A.chunks = pl.chunks;
    A.ctas = pl.ctas;
    const auto kernel = pl.packs == 8 ? distill_kernel<T, 8, MODE> : pl.packs == 4 ? distill_kernel<T, 4, MODE> : distill_kernel<T, 2, MODE>;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)pl.ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(N * pl.ctas));
    cfg.blockDim = dim3((unsigned)pl.threads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return (int)cudaLaunchKernelEx(&cfg, kernel, A);
}

template <int MODE>
int run(const distill_params_t* p, const DistillArgs& A, cudaStream_t st)
{
    if (distill_walks_rows(p)) return launch_distill_rows(p, A, MODE, st);
    const Plan pl = plan_of(p);
    return p->dtype == GDN_F32    ? launch<float, MODE>(A, pl, p->N, st)
           : p->dtype == GDN_BF16 ? launch<__nv_bfloat16, MODE>(A, pl, p->N, st)
                                  : launch<__half, MODE>(A, pl, p->N, st);
}

struct Buffer {
    const void* ptr;
    size_t n;
};

int check_buffers(const distill_params_t* p, const void* logits, const int32_t* indices, const void* teacher, const float* lse_in, const float* dloss,
                  const Buffer (&small)[2], void* dlogits)
{
    const size_t es = elem_size(p->dtype), ts = elem_size(p->teacher_dtype), N = (size_t)p->N, K = (size_t)p->K;
    if (!logits || (K && (!indices || !teacher))) return fail(GDN_ERR_INVALID_ARG, "distill: NULL pointer");
    if ((uintptr_t)logits % es || (uintptr_t)dlogits % es || (uintptr_t)indices % 4 || (uintptr_t)teacher % ts || (uintptr_t)lse_in % 4 || (uintptr_t)dloss % 4 ||
        (uintptr_t)small[0].ptr % 4 || (uintptr_t)small[1].ptr % 4)
        return fail(GDN_ERR_INVALID_ARG, "distill: a pointer is not aligned to its element");
    const size_t n_x = ((N - 1) * (size_t)p->row_stride + (size_t)p->V) * es, n_d = ((N - 1) * (size_t)p->d_stride + (size_t)p->V) * es;
    const Buffer in[] = {{logits, n_x}, {indices, N * K * 4}, {teacher, N * K * ts}, {lse_in, N * 4}, {dloss, N * 4}};
    const Buffer out[] = {small[0], small[1], {dlogits, n_d}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 5; ++j) {
            if (i == 2 && j == 0 && dlogits == logits && p->row_stride == p->d_stride) continue;  // in place
            if (overlap(out[i].ptr, out[i].n, in[j].ptr, in[j].n)) return fail(GDN_ERR_ALIAS, "distill: an output overlaps an input");
        }
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].ptr, out[i].n, out[j].ptr, out[j].n)) return fail(GDN_ERR_ALIAS, "distill: outputs overlap");
    }
    return GDN_OK;
}

DistillArgs args_of(const distill_params_t* p, const void* logits, const int32_t* indices, const void* teacher, const float* dloss, void* dlogits)
{
    DistillArgs A{};
    A.logits = logits; A.indices = indices; A.teacher = teacher; A.dloss = dloss; A.dlogits = dlogits;
    A.row_stride = p->row_stride; A.d_stride = p->d_stride;
    A.V = (int)p->V; A.K = (int)p->K; A.teacher_dtype = p->teacher_dtype;
    A.inv_tau = (float)(1.0 / (double)p->temperature);
    A.L = (float)(1.4426950408889634 / (double)p->temperature);
    return A;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" int distill_forward(const distill_params_t* p, const void* logits, const int32_t* indices, const void* teacher, float* loss,
                               float* lse, const float* dloss, void* dlogits, void* stream)
{
    int st = check(p);
    if (st != GDN_OK || p->N == 0) return st;
    if (!loss || !lse || !dloss != !dlogits) return fail(GDN_ERR_INVALID_ARG, "distill_forward: NULL pointer, or one of dloss and dlogits without the other");
    const size_t n = (size_t)p->N * 4;
    st = check_buffers(p, logits, indices, teacher, nullptr, dloss, {{loss, n}, {lse, n}}, dlogits);
    if (st != GDN_OK) return st;
    DistillArgs A = args_of(p, logits, indices, teacher, dloss, dlogits);
    A.loss = loss;
    A.lse = lse;
    const int e = dlogits ? run<kBoth>(p, A, (cudaStream_t)stream) : run<kLoss>(p, A, (cudaStream_t)stream);
    return e ? cuda_fail(e, "distill_forward launch") : GDN_OK;
}

extern "C" int distill_backward(const distill_params_t* p, const void* logits, const int32_t* indices, const void* teacher, const float* lse,
                                const float* dloss, void* dlogits, void* stream)
{
    int st = check(p);
    if (st != GDN_OK || p->N == 0) return st;
    if (!lse || !dloss || !dlogits) return fail(GDN_ERR_INVALID_ARG, "distill_backward: NULL pointer");
    st = check_buffers(p, logits, indices, teacher, lse, dloss, {{nullptr, 0}, {nullptr, 0}}, dlogits);
    if (st != GDN_OK) return st;
    DistillArgs A = args_of(p, logits, indices, teacher, dloss, dlogits);
    A.lse_in = lse;
    const int e = run<kGradient>(p, A, (cudaStream_t)stream);
    return e ? cuda_fail(e, "distill_backward launch") : GDN_OK;
}
