// gdn_decode.cu -- the gated delta rule's serving form (include/gdn_decode.h): the recurrence
// over a pool of states, a few tokens a sequence.
//
// Mathematics.  Only rows of the state meet the tokens, M[j] . k and M[j] . q, so every row of a
// state goes its own way: a warp takes 4 RT rows, keeps them in registers over the sequence's tokens, and
// reads and writes them once.  Both dots are taken of the state before the token, u = M k, o = M q, and
//     delta = beta (v - a u),   y = scale (a o + delta (k . q)),   M <- a M + delta k^T
// so that one pass over the row and one exchange between lanes serve a token (the KDA gate puts
// its a into k and q: M (a k), M (a q)).
//
// What bounds it: the states' bytes, 8 S_k S_v a head against 7 S_k S_v flops a token.  So the
// layout follows the reads: 8 lanes a row, each with float4 blocks 32 columns apart (whole 128-byte
// lines), 4 rows across the warp, all of a warp's state in flight before its first use.  The warps of
// a CTA share one head: each widens (and for KDA exponentiates) one of the next W tokens into
// shared memory for all of them, and one barrier serves W tokens.
//
// Measured at 48 heads of 128 (16 key heads, bf16): 64 sequences' next tokens 63 us, 6.4 TB/s of 6.7 for a copy;
// 200 sequences of up to 5 tokens, KDA, 204 us, 6.3 TB/s (four CTAs an SM; three 233 us; every warp
// widening its own tokens 248 us; every lane 643 us); one sequence 3.1 us.  Many tokens on small heads
// are bound by the fp32 pipe and by the longest sequence: 60 sequences of 16 tokens, 4 heads of 64, 9.6 us.
#include <climits>
#include <cstdio>

#include "../../include/gdn_decode.h"
#include "gdn_device.cuh"
#include "gdn_elem.cuh"
#include "gdn_f32x2.cuh"
#include "gdn_launch.cuh"

namespace gdn {
namespace {

// Bit 0: gdn_decode met a bad slot or token range; bit 1: gdn_states_move a bad slot.
__device__ int g_decode_status;

struct DecodeArgs {
    const void *q, *k, *v, *g, *beta;
    const int* cu;
    float* pool;
    const int *slot_in, *slot_out;
    void* y;
    long long slot_stride, qs0, qs1, ks0, ks1, vs0, vs1;
    int T, n_tok, n_slots, H_k, H_v, SK, SV;
    int gate_dtype, y_dtype, vec, vec_g;
    float scale;
};

// Four consecutive gates as fp32.
__device__ __forceinline__ float4 ld_gate4(const void* p, long long i, int dtype, bool vec)
{
    if (vec && dtype == GDN_F32) return ld_plain(reinterpret_cast<const float4*>((const float*)p + i));
    return make_float4(ld_any(p, i, dtype), ld_any(p, i + 1, dtype), ld_any(p, i + 2, dtype), ld_any(p, i + 3, dtype));
}

// A token's row vectors and numbers in fp32, for all warps of a CTA: what the dots take of the state (k, q; times
// the gate for KDA), for KDA also k and the gate itself, the CTA's rows of v, and {exp g, beta, k . q}.
template <int NV, int RT, bool KDA>
struct Staged {
    float4 vec[KDA ? 4 : 2][8 * NV];
    float v[16 * RT];
    float4 num;
};

// A lane's share of one token as it arrives.
template <typename T, int NV, int RT, bool KDA>
struct Token {
    static constexpr int SHARE = (32 * NV + 127) / 128, ROWS = (16 * RT + 31) / 32;
    Pack<T, 4> q[SHARE], k[SHARE];
    float4 g[SHARE];  // scalar gate: g[0].x
    T v[ROWS];
    float beta;
};

template <typename T, int NV, int RT, bool KDA>
__device__ __forceinline__ void load_token(Token<T, NV, RT, KDA>& x, const DecodeArgs& A, const T* q, const T* k, const T* v, int rows,
                                           long long row, int h, int lane)
{
    const long long gh = row * A.H_v + h;
    x.beta = ld_any(A.beta, gh, A.gate_dtype);
    if (!KDA) x.g[0].x = ld_any(A.g, gh, A.gate_dtype);
#pragma unroll
    for (int s = 0; s < x.ROWS; ++s)
        if (32 * s + lane < rows) x.v[s] = ld_plain(v + row * A.vs0 + 32 * s + lane);
#pragma unroll
    for (int s = 0; s < x.SHARE; ++s) {
        const int c = 128 * s + 4 * lane;
        if (c < A.SK) {
            x.k[s] = ld_pack<T, 4>(k + row * A.ks0 + c, A.vec);
            x.q[s] = ld_pack<T, 4>(q + row * A.qs0 + c, A.vec);
            if (KDA) x.g[s] = ld_gate4(A.g, gh * A.SK + c, A.gate_dtype, A.vec_g);
        }
    }
}

// One warp widens (and for KDA exponentiates) a token into shared memory.
template <typename T, int NV, int RT, bool KDA>
__device__ __forceinline__ void stage_token(Staged<NV, RT, KDA>& S, const Token<T, NV, RT, KDA>& x, const DecodeArgs& A, int rows, int lane)
{
    float kq = 0.f;
#pragma unroll
    for (int s = 0; s < x.SHARE; ++s) {
        const int c = 128 * s + 4 * lane;
        float4 k = make_float4(0.f, 0.f, 0.f, 0.f), q = k, a = k;
        if (c < A.SK) {
            k = make_float4(x.k[s].get(0), x.k[s].get(1), x.k[s].get(2), x.k[s].get(3));
            q = make_float4(x.q[s].get(0), x.q[s].get(1), x.q[s].get(2), x.q[s].get(3));
            if (KDA) a = make_float4(expf(x.g[s].x), expf(x.g[s].y), expf(x.g[s].z), expf(x.g[s].w));
        }
        kq += (k.x * q.x + k.y * q.y) + (k.z * q.z + k.w * q.w);
        if (c < 32 * NV) {
            if (KDA) {
                S.vec[KDA ? 2 : 0][c / 4] = k;
                S.vec[KDA ? 3 : 0][c / 4] = a;
                k = make_float4(k.x * a.x, k.y * a.y, k.z * a.z, k.w * a.w);
                q = make_float4(q.x * a.x, q.y * a.y, q.z * a.z, q.w * a.w);
            }
            S.vec[0][c / 4] = k;
            S.vec[1][c / 4] = q;
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) kq += __shfl_xor_sync(kFull, kq, o);
#pragma unroll
    for (int s = 0; s < x.ROWS; ++s)
        if (32 * s + lane < rows) S.v[32 * s + lane] = to_f32(x.v[s]);
    if (lane == 0) S.num = make_float4(KDA ? 1.f : expf(x.g[0].x), x.beta, kq, 0.f);
}

// One CTA of W <= 4 warps: 4 RT W rows of one head's state.  RT: rows of a lane; NV: its float4 blocks of a row.
template <typename T, int NV, int RT, bool KDA>
__global__ void __launch_bounds__(128, RT * NV >= 16 ? 4 : RT * NV >= 8 ? 5 : 6) gdn_decode_kernel(const DecodeArgs A)
{
    __shared__ Staged<NV, RT, KDA> staged[2][4];  // W tokens, while the next W arrive
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5, cl = lane & 7, grp = lane >> 3;
    const int rows = 4 * RT * W;  // of the CTA
    const unsigned per_head = A.SV / rows, nh = blockIdx.x / per_head;
    const int first = (int)(blockIdx.x - nh * per_head) * rows, row0 = first + warp * 4 * RT;
    const int n = nh / A.H_v, h = nh - n * A.H_v;

    begin_after();
    const int s_in = ld_plain(A.slot_in + n), s_out = ld_plain(A.slot_out + n);
    long long lo, hi;
    if (A.cu) {
        lo = ld_plain(A.cu + n);
        hi = ld_plain(A.cu + n + 1);
    } else {
        lo = (long long)n * A.T;
        hi = lo + A.T;
    }
    if (s_in < -1 || s_in >= A.n_slots || s_out < -1 || s_out >= A.n_slots || lo < 0 || hi < lo || hi > A.n_tok) {
        if (threadIdx.x == 0) atomicOr(&g_decode_status, 1);
        return;
    }
    const int hk = h % A.H_k;
    const T *qh = (const T*)A.q + hk * A.qs1, *kh = (const T*)A.k + hk * A.ks1, *vh = (const T*)A.v + h * A.vs1 + first;
    Token<T, NV, RT, KDA> x;
    if (lo + warp < hi) load_token<T, NV, RT, KDA>(x, A, qh, kh, vh, rows, lo + warp, h, lane);

    // rows row0 + grp RT + r of the state, r < RT
    const long long at = ((long long)h * A.SV + row0 + grp * RT) * A.SK;
    f2 m[RT][NV][2];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int b = 0; b < NV; ++b) {
            const int c = 32 * b + 4 * cl;
            ulonglong2 v = make_ulonglong2(0, 0);
            if (s_in >= 0 && c < A.SK)
                v = *reinterpret_cast<const ulonglong2*>(A.pool + s_in * A.slot_stride + at + r * A.SK + c);
            m[r][b][0] = v.x;
            m[r][b][1] = v.y;
        }

    // After the exchange between a row's 8 lanes, lanes 0-3 hold u and lanes 4-7 o; row mine of the RT.
    constexpr int kShare = 4 / RT;  // lanes that hold the same sum
    const int mine = (cl & 3) / kShare;
    const int j = row0 + grp * RT + mine;

    if (lo + warp < hi) stage_token<T, NV, RT, KDA>(staged[0][warp], x, A, rows, lane);
    if (lo + W + warp < hi) load_token<T, NV, RT, KDA>(x, A, qh, kh, vh, rows, lo + W + warp, h, lane);
    const bool writes = cl >= 4 && (cl & (kShare - 1)) == 0;
    const int y_shift = A.y_dtype == GDN_F32 ? 2 : 1;
    char* y = (char*)A.y + (((lo * A.H_v + h) * A.SV + j) << y_shift);
    const long long y_step = (long long)A.H_v * A.SV << y_shift;
    int set = 0;
    for (long long t0 = lo; t0 < hi; t0 += W, set ^= 1) {
        __syncthreads();
        // the tokens after these W, staged by the warps while they are in them
        if (t0 + W + warp < hi) {
            stage_token<T, NV, RT, KDA>(staged[set ^ 1][warp], x, A, rows, lane);
            if (t0 + 2 * W + warp < hi) load_token<T, NV, RT, KDA>(x, A, qh, kh, vh, rows, t0 + 2 * W + warp, h, lane);
        }
        const int now = hi - t0 < W ? (int)(hi - t0) : W;
        for (int i = 0; i < now; ++i) {
            const Staged<NV, RT, KDA>& S = staged[set][i];
            const float4 num = S.num;
            const float vj = S.v[j - first];
            float s[2 * RT];
            {
                f2 u2[RT], o2[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) u2[r] = o2[r] = 0;
#pragma unroll
                for (int b = 0; b < NV; ++b) {
                    const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(&S.vec[0][8 * b + cl]);
                    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&S.vec[1][8 * b + cl]);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        u2[r] = fma2(m[r][b][0], k.x, u2[r]);
                        o2[r] = fma2(m[r][b][0], q.x, o2[r]);
                        u2[r] = fma2(m[r][b][1], k.y, u2[r]);
                        o2[r] = fma2(m[r][b][1], q.y, o2[r]);
                    }
                }
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    s[r] = sum2(u2[r]);
                    s[RT + r] = sum2(o2[r]);
                }
            }
            // reduce-scatter of the 2 RT sums over the 8 lanes, then a butterfly over the lanes that share one
#pragma unroll
            for (int n2 = RT, bit = 4; n2 >= 1; n2 >>= 1, bit >>= 1) {
                const bool up = (cl & bit) != 0;
#pragma unroll
                for (int e = 0; e < n2; ++e) {
                    const float send = up ? s[e] : s[n2 + e], keep = up ? s[n2 + e] : s[e];
                    s[e] = keep + __shfl_xor_sync(kFull, send, bit);
                }
            }
#pragma unroll
            for (int bit = kShare / 2; bit >= 1; bit >>= 1) s[0] += __shfl_xor_sync(kFull, s[0], bit);
            const float sum = KDA ? s[0] : num.x * s[0];
            float delta = num.y * (vj - sum);  // on lanes 0-3
            float d[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) d[r] = __shfl_sync(kFull, delta, (lane & 24) + r * kShare);
            delta = __shfl_xor_sync(kFull, delta, 4);
            if (writes) st_any(y, 0, A.y_dtype, A.scale * fmaf(delta, num.z, sum));
            y += y_step;
            const f2 as2 = pack2(num.x, num.x);
#pragma unroll
            for (int b = 0; b < NV; ++b) {
                const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(&S.vec[KDA ? 2 : 0][8 * b + cl]);
                ulonglong2 a = make_ulonglong2(as2, as2);
                if (KDA) a = *reinterpret_cast<const ulonglong2*>(&S.vec[KDA ? 3 : 0][8 * b + cl]);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const f2 dd = pack2(d[r], d[r]);
                    m[r][b][0] = fma2(k.x, dd, mul2(m[r][b][0], a.x));
                    m[r][b][1] = fma2(k.y, dd, mul2(m[r][b][1], a.y));
                }
            }
        }
    }

    if (s_out < 0) return;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int b = 0; b < NV; ++b) {
            const int c = 32 * b + 4 * cl;
            if (c < A.SK)
                *reinterpret_cast<ulonglong2*>(A.pool + s_out * A.slot_stride + at + r * A.SK + c) =
                    make_ulonglong2(m[r][b][0], m[r][b][1]);
        }
}

template <typename T, int NV, int RT>
int launch_decode_g(const DecodeArgs& A, long long heads, bool kda, cudaStream_t st)
{
    const int groups = A.SV / (4 * RT);  // warps' rows of a head
    int W = 4;
    while (groups % W != 0) --W;
    const unsigned ctas = (unsigned)(heads * (groups / W));
    return launch_after(kda ? gdn_decode_kernel<T, NV, RT, true> : gdn_decode_kernel<T, NV, RT, false>, ctas, 32 * W, 0, st, A);
}

template <typename T>
int launch_decode_t(const DecodeArgs& A, long long heads, bool kda, cudaStream_t st)
{
    // Few heads are spread over more warps of one row a lane; many take more rows a lane, so that a token's
    // q and k serve them all.  Both sides, one row against four a lane: 48 heads of 128, 1 sequence 3.1 and
    // 3.2 us, 4 sequences 6.2 and 5.5, 8 sequences 13.7 and 10.9; 8 x 4 heads of 64, 16 tokens, 6.9 and 8.0.
    const bool wide = heads * A.SV >= 16 * 4 * kNumSMs;
    if (A.SK <= 32) return wide ? launch_decode_g<T, 1, 4>(A, heads, kda, st) : launch_decode_g<T, 1, 1>(A, heads, kda, st);
    if (A.SK == 64) return wide ? launch_decode_g<T, 2, 4>(A, heads, kda, st) : launch_decode_g<T, 2, 1>(A, heads, kda, st);
    if (A.SK == 128) return wide ? launch_decode_g<T, 4, 4>(A, heads, kda, st) : launch_decode_g<T, 4, 1>(A, heads, kda, st);
    return wide ? launch_decode_g<T, 8, 2>(A, heads, kda, st) : launch_decode_g<T, 8, 1>(A, heads, kda, st);
}

gdn_status_t fail(gdn_status_t s, const char* msg)
{
    set_last_error(msg);
    return s;
}

gdn_status_t cuda_fail(int e, const char* what)
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

// Bytes that rows of H heads of S elements reach over.
size_t span(int64_t rows, int64_t H, int64_t S, const int64_t s[2], size_t es)
{
    return rows < 1 ? 0 : (size_t)((rows - 1) * s[0] + (H - 1) * s[1] + S) * es;
}

gdn_status_t check_decode(const gdn_decode_params_t* p)
{
    if (!p) return fail(GDN_ERR_INVALID_ARG, "gdn_decode: params is NULL");
    if (p->n_seq < 0 || p->T < 0 || p->n_tok < 0 || p->n_slots < 0)
        return fail(GDN_ERR_INVALID_ARG, "gdn_decode: negative n_seq, T, n_tok or n_slots");
    if (p->H_k < 1 || p->H_v < 1 || p->S_k < 1 || p->S_v < 1)
        return fail(GDN_ERR_INVALID_ARG, "gdn_decode: heads and head sizes must be >= 1");
    if (p->H_v % p->H_k != 0) return fail(GDN_ERR_INVALID_ARG, "gdn_decode: H_v is not a multiple of H_k");
    if (p->gate != GDN_GATE_SCALAR && p->gate != GDN_GATE_KDA) return fail(GDN_ERR_INVALID_ARG, "gdn_decode: unknown gate kind");
    if (!known_dtype(p->in_dtype) || !known_dtype(p->gate_dtype) || !known_dtype(p->y_dtype))
        return fail(GDN_ERR_INVALID_ARG, "gdn_decode: unknown dtype");
    for (int i = 0; i < 2; ++i)
        if (p->q_s[i] < 0 || p->k_s[i] < 0 || p->v_s[i] < 0) return fail(GDN_ERR_INVALID_ARG, "gdn_decode: negative stride");
    if (p->S_k != 16 && p->S_k != 32 && p->S_k != 64 && p->S_k != 128 && p->S_k != 256)
        return fail(GDN_ERR_UNSUPPORTED, "gdn_decode: S_k must be 16, 32, 64, 128 or 256");
    if (p->S_v % 16 != 0 || p->S_v > 256) return fail(GDN_ERR_UNSUPPORTED, "gdn_decode: S_v must be a multiple of 16 up to 256");
    if (p->H_v > 65535 || p->n_tok > INT_MAX || p->T > INT_MAX || p->n_slots > INT_MAX ||
        p->n_seq > (int64_t)INT_MAX / (p->H_v * (p->S_v / 4)))
        return fail(GDN_ERR_UNSUPPORTED, "gdn_decode: sizes beyond the kernel's index range");
    if (p->slot_stride < p->H_v * p->S_v * p->S_k || p->slot_stride % 4 != 0)
        return fail(GDN_ERR_INVALID_ARG, "gdn_decode: slot_stride must be a multiple of 4 of at least H_v S_v S_k");
    return GDN_OK;
}

bool vec4(const void* ptr, const int64_t s[2], size_t es)
{
    return (uintptr_t)ptr % (4 * es) == 0 && s[0] % 4 == 0 && s[1] % 4 == 0;
}

}  // namespace

int decode_take_status(void* stream, int* status)
{
    cudaStream_t s = (cudaStream_t)stream;
    int v = 0;
    int e = (int)cudaMemcpyFromSymbolAsync(&v, g_decode_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (!e) e = (int)cudaStreamSynchronize(s);
    if (e) return e;
    if (v) {
        const int zero = 0;
        e = (int)cudaMemcpyToSymbolAsync(g_decode_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
        if (!e) e = (int)cudaStreamSynchronize(s);
    }
    *status = v;
    return e;
}

}  // namespace gdn

using namespace gdn;

extern "C" gdn_status_t gdn_decode_supported(const gdn_decode_params_t* p) { return check_decode(p); }

extern "C" gdn_status_t gdn_decode(const gdn_decode_params_t* p, const void* q, const void* k, const void* v, const void* g,
                                   const void* beta, const int32_t* cu_tokens, float* pool, const int32_t* slot_in,
                                   const int32_t* slot_out, void* y, void* stream)
{
    const gdn_status_t st = check_decode(p);
    if (st != GDN_OK) return st;
    if (!cu_tokens && p->n_tok != p->n_seq * p->T)
        return fail(GDN_ERR_INVALID_ARG, "gdn_decode: without cu_tokens, n_tok must be n_seq T");
    if (p->n_seq == 0) return GDN_OK;
    if (!slot_in || !slot_out || (p->n_slots > 0 && !pool) || (p->n_tok > 0 && (!q || !k || !v || !g || !beta || !y)))
        return fail(GDN_ERR_INVALID_ARG, "gdn_decode: NULL pointer");
    const size_t es = elem_size(p->in_dtype), gs = elem_size(p->gate_dtype), ys = elem_size(p->y_dtype);
    if ((uintptr_t)pool % 16 != 0) return fail(GDN_ERR_INVALID_ARG, "gdn_decode: the pool must be 16-byte aligned");
    if ((uintptr_t)q % es || (uintptr_t)k % es || (uintptr_t)v % es || (uintptr_t)g % gs || (uintptr_t)beta % gs ||
        (uintptr_t)y % ys || (uintptr_t)slot_in % 4 || (uintptr_t)slot_out % 4 || (uintptr_t)cu_tokens % 4)
        return fail(GDN_ERR_INVALID_ARG, "gdn_decode: a pointer is not aligned to its element");
    const bool kda = p->gate == GDN_GATE_KDA;
    const size_t n_pool = p->n_slots > 0 ? (size_t)((p->n_slots - 1) * p->slot_stride + p->H_v * p->S_v * p->S_k) * 4 : 0;
    const size_t n_y = (size_t)(p->n_tok * p->H_v * p->S_v) * ys, n_b = (size_t)(p->n_tok * p->H_v) * gs;
    const struct { const void* ptr; size_t n; } in[] = {
        {q, span(p->n_tok, p->H_k, p->S_k, p->q_s, es)}, {k, span(p->n_tok, p->H_k, p->S_k, p->k_s, es)},
        {v, span(p->n_tok, p->H_v, p->S_v, p->v_s, es)}, {g, n_b * (kda ? (size_t)p->S_k : 1)}, {beta, n_b},
        {cu_tokens, (size_t)(p->n_seq + 1) * 4}, {slot_in, (size_t)p->n_seq * 4}, {slot_out, (size_t)p->n_seq * 4}};
    for (const auto& i : in)
        if (overlap(i.ptr, i.n, y, n_y) || overlap(i.ptr, i.n, pool, n_pool))
            return fail(GDN_ERR_ALIAS, "gdn_decode: y or the pool overlaps an input");
    if (overlap(y, n_y, pool, n_pool)) return fail(GDN_ERR_ALIAS, "gdn_decode: y overlaps the pool");

    DecodeArgs A{};
    A.q = q; A.k = k; A.v = v; A.g = g; A.beta = beta; A.cu = cu_tokens; A.pool = pool;
    A.slot_in = slot_in; A.slot_out = slot_out; A.y = y;
    A.slot_stride = p->slot_stride;
    A.qs0 = p->q_s[0]; A.qs1 = p->q_s[1]; A.ks0 = p->k_s[0]; A.ks1 = p->k_s[1]; A.vs0 = p->v_s[0]; A.vs1 = p->v_s[1];
    A.T = (int)p->T; A.n_tok = (int)p->n_tok; A.n_slots = (int)p->n_slots;
    A.H_k = (int)p->H_k; A.H_v = (int)p->H_v; A.SK = (int)p->S_k; A.SV = (int)p->S_v;
    A.gate_dtype = p->gate_dtype; A.y_dtype = p->y_dtype; A.scale = p->scale;
    A.vec = vec4(q, p->q_s, es) && vec4(k, p->k_s, es);
    A.vec_g = (uintptr_t)g % 16 == 0;
    const long long heads = p->n_seq * p->H_v;
    cudaStream_t s = (cudaStream_t)stream;
    const int e = p->in_dtype == GDN_F32    ? launch_decode_t<float>(A, heads, kda, s)
                  : p->in_dtype == GDN_BF16 ? launch_decode_t<__nv_bfloat16>(A, heads, kda, s)
                                            : launch_decode_t<__half>(A, heads, kda, s);
    return e ? cuda_fail(e, "gdn_decode launch") : GDN_OK;
}

namespace gdn {
namespace {

constexpr int kMostGroup = 1024, kLeastPiece = 128, kMostGroupBytes = kMostGroup * kLeastPiece;  // of larger groups

struct MoveArgs {
    char* pool;
    const int *src, *dst;
    long long layer_stride, slot_stride, state_bytes;
    int n_slots, n_moves, group, piece;  // piece: bytes of a state that one CTA moves, for every move of its group
    unsigned pieces, groups;
};

__device__ __forceinline__ bool bad_move(const MoveArgs& A, int s, int d) { return s < -1 || s >= A.n_slots || d < -1 || d >= A.n_slots; }

// Groups of up to G moves, without shared memory or barriers: a thread takes the same 16 bytes (P times) of every
// slot of its group, and nobody else touches those, so that having read all sources before it writes any
// destination is all that simultaneous takes.  A source of several destinations is read from DRAM once:
// the thread's own later reads of it find it in L1.  Bytes bound it: 64 states of 3 MB copied in two layers take
// 119 us, 6.75 TB/s, as do groups of 2 and of 16; one 16-byte place a thread (four without a group) is enough.
template <int G, int P>
__global__ void __launch_bounds__(256) gdn_states_move_kernel(const MoveArgs A)
{
    __shared__ long long from[G], to[G];  // bytes into the pool; from -1: zeros, -2: nothing to do
    const unsigned pc = blockIdx.x % A.pieces, gl = blockIdx.x / A.pieces;
    const unsigned gr = gl % A.groups, layer = gl / A.groups;
    const int nm = min(A.group, A.n_moves - (int)gr * A.group);
    begin_after();
    if (threadIdx.x < G) {
        long long f = -2, t = 0;
        if ((int)threadIdx.x < nm) {
            const int s = ld_plain(A.src + gr * A.group + threadIdx.x), d = ld_plain(A.dst + gr * A.group + threadIdx.x);
            if (bad_move(A, s, d)) {
                if (pc == 0 && layer == 0) atomicOr(&g_decode_status, 2);
            } else if (d >= 0 && s != d) {
                f = s < 0 ? -1 : layer * A.layer_stride + s * A.slot_stride;
                t = layer * A.layer_stride + d * A.slot_stride;
            }
        }
        from[threadIdx.x] = f;
        to[threadIdx.x] = t;
    }
    __syncthreads();
    const long long at = (long long)pc * A.piece + threadIdx.x * 16;
    uint4 v[G][P];
#pragma unroll
    for (int m = 0; m < G; ++m) {
        const long long f = from[m];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            v[m][p] = make_uint4(0, 0, 0, 0);
            if (f >= 0 && at + p * 4096 < A.state_bytes) v[m][p] = *reinterpret_cast<const uint4*>(A.pool + f + at + p * 4096);
        }
    }
#pragma unroll
    for (int m = 0; m < G; ++m) {
        if (from[m] < -1) continue;
        char* t = A.pool + to[m];
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (at + p * 4096 < A.state_bytes) *reinterpret_cast<uint4*>(t + at + p * 4096) = v[m][p];
    }
}

// Larger groups: every source's piece is in shared memory before the first destination is written.
__global__ void __launch_bounds__(256) gdn_states_move_large_kernel(const MoveArgs A)
{
    extern __shared__ uint4 buf[];
    const unsigned pc = blockIdx.x % A.pieces, gl = blockIdx.x / A.pieces;
    const unsigned gr = gl % A.groups, layer = gl / A.groups;
    const long long at = (long long)pc * A.piece;
    const int bytes = (int)(A.state_bytes - at < A.piece ? A.state_bytes - at : A.piece);
    const int n16 = bytes / 16, per = A.piece / 16;
    const int m0 = gr * A.group, nm = A.n_moves - m0 < A.group ? A.n_moves - m0 : A.group;
    char* base = A.pool + layer * A.layer_stride + at;
    begin_after();
    for (int i = threadIdx.x; i < nm * n16; i += blockDim.x) {
        const int m = i / n16, e = i - m * n16;
        const int s = ld_plain(A.src + m0 + m), d = ld_plain(A.dst + m0 + m);
        if (bad_move(A, s, d)) {
            if (e == 0) atomicOr(&g_decode_status, 2);
            continue;
        }
        if (d < 0 || s == d) continue;
        buf[m * per + e] = s < 0 ? make_uint4(0, 0, 0, 0) : reinterpret_cast<const uint4*>(base + s * A.slot_stride)[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nm * n16; i += blockDim.x) {
        const int m = i / n16, e = i - m * n16;
        const int s = ld_plain(A.src + m0 + m), d = ld_plain(A.dst + m0 + m);
        if (bad_move(A, s, d) || d < 0 || s == d) continue;
        reinterpret_cast<uint4*>(base + d * A.slot_stride)[e] = buf[m * per + e];
    }
}

template <int G, int P>
int launch_move(const MoveArgs& A, unsigned ctas, cudaStream_t st)
{
    return launch_after(gdn_states_move_kernel<G, P>, ctas, 256, 0, st, A);
}

}  // namespace
}  // namespace gdn

extern "C" gdn_status_t gdn_states_move(void* pool, int64_t n_layers, int64_t layer_stride, int64_t n_slots,
                                        int64_t slot_stride, int64_t state_bytes, const int32_t* src, const int32_t* dst,
                                        int64_t n_moves, int64_t group, void* stream)
{
    if (n_layers < 0 || n_slots < 0 || state_bytes < 0 || n_moves < 0 || layer_stride < 0 || slot_stride < 0 || group < 1)
        return fail(GDN_ERR_INVALID_ARG, "gdn_states_move: negative size or stride, or group < 1");
    if (group > n_moves) group = n_moves > 0 ? n_moves : 1;
    if (group > kMostGroup) return fail(GDN_ERR_UNSUPPORTED, "gdn_states_move: more than 1024 moves in a group");
    if (n_layers == 0 || n_moves == 0 || state_bytes == 0 || n_slots == 0) return GDN_OK;
    if (!pool || !src || !dst) return fail(GDN_ERR_INVALID_ARG, "gdn_states_move: NULL pointer");
    if ((uintptr_t)pool % 16 || layer_stride % 16 || slot_stride % 16 || state_bytes % 16 || (uintptr_t)src % 4 || (uintptr_t)dst % 4)
        return fail(GDN_ERR_INVALID_ARG, "gdn_states_move: the pool, its strides and state_bytes must be multiples of 16 bytes");
    if ((n_slots > 1 && slot_stride < state_bytes) || n_slots > INT_MAX || n_moves > INT_MAX)
        return fail(GDN_ERR_INVALID_ARG, "gdn_states_move: slots overlap, or too many of them");
    // layers lie one after the other, or inside one another's slots ([slot][layer] order)
    const int64_t slots_span = (n_slots - 1) * slot_stride + state_bytes, layers_span = (n_layers - 1) * layer_stride + state_bytes;
    if (n_layers > 1 && layer_stride < slots_span && !(layer_stride >= state_bytes && (n_slots == 1 || slot_stride >= layers_span)))
        return fail(GDN_ERR_INVALID_ARG, "gdn_states_move: layers overlap");
    const size_t n_pool = (size_t)((n_layers - 1) * layer_stride + slots_span);
    if (overlap(src, (size_t)n_moves * 4, pool, n_pool) || overlap(dst, (size_t)n_moves * 4, pool, n_pool))
        return fail(GDN_ERR_ALIAS, "gdn_states_move: src or dst inside the pool");

    MoveArgs A{};
    A.pool = (char*)pool; A.src = src; A.dst = dst;
    A.layer_stride = layer_stride; A.slot_stride = slot_stride; A.state_bytes = state_bytes;
    A.n_slots = (int)n_slots; A.n_moves = (int)n_moves; A.group = (int)group;
    const int G = group <= 2 ? (int)group : group <= 4 ? 4 : group <= 8 ? 8 : 16;
    int64_t piece;
    if (group <= 16) {
        piece = 4096 * (G == 1 ? 4 : 1);  // 16 bytes of 256 threads, P times
    } else {
        piece = 32 * 1024 / group / 16 * 16;
        if (piece < kLeastPiece) piece = kLeastPiece;
        if (piece > state_bytes) piece = state_bytes;
    }
    A.piece = (int)piece;
    A.pieces = (unsigned)((state_bytes + piece - 1) / piece);
    A.groups = (unsigned)((n_moves + group - 1) / group);
    const int64_t ctas = (int64_t)A.pieces * A.groups * n_layers;
    if ((state_bytes + piece - 1) / piece > INT_MAX || ctas > INT_MAX)
        return fail(GDN_ERR_UNSUPPORTED, "gdn_states_move: too many pieces for one launch");
    cudaStream_t st = (cudaStream_t)stream;
    int e = 0;
    if (G == 1 && group <= 16) e = launch_move<1, 4>(A, (unsigned)ctas, st);
    else if (G == 2 && group <= 16) e = launch_move<2, 1>(A, (unsigned)ctas, st);
    else if (G == 4 && group <= 16) e = launch_move<4, 1>(A, (unsigned)ctas, st);
    else if (G == 8 && group <= 16) e = launch_move<8, 1>(A, (unsigned)ctas, st);
    else if (group <= 16) e = launch_move<16, 1>(A, (unsigned)ctas, st);
    else {
        const size_t smem = (size_t)(piece * group);
        // the limit is the kernel's, not the call's: every call sets the same, so that none lowers another thread's
        if (smem > 40 * 1024)
            e = (int)cudaFuncSetAttribute(gdn_states_move_large_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostGroupBytes);
        if (!e) e = launch_after(gdn_states_move_large_kernel, (unsigned)ctas, 256, smem, st, A);
    }
    return e ? cuda_fail(e, "gdn_states_move launch") : GDN_OK;
}
