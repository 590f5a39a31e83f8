// la_token.cu -- linear attention's token form (include/la.h): the core of la_internal.h token by token.
//
// Every row of a state goes its own way: S[j] <- a S[j] + cs z_j y, out_j = co S[j] . x.  So a warp keeps 4 RT rows in
// registers over the sequence's tokens, 8 lanes a row, each with float4 blocks 32 columns apart (whole 128-byte
// lines), and reads and writes a state once.  The warps of a CTA share one head: each widens one of the next W tokens
// into shared memory for all of them, and one barrier serves W tokens.
//
// Of the backward pass's dq and dk, CTAs of a head may share a sequence by segments (launch_la_tokens).
//
// What bounds it: for a token or a few the states' bytes, 8 S_k S_v a head against 4 S_k S_v flops a token (64 sequences of 48 heads
// of 128, one token: 65 us, 6.2 TB/s, 93 % of the copy rate); for many tokens the chain of tokens, 0.5 us each (32 heads of 128, 32 tokens: 23 us); for
// the smallest calls latency (one sequence: 7 us alone and cold, two dependent loads, a barrier and cold instructions).
#include <type_traits>

#include "gdn_device.cuh"
#include "gdn_elem.cuh"
#include "gdn_launch.cuh"
#include "la_internal.h"

namespace gdn {
namespace {

__device__ int g_la_token_status;

// How a state decays: m <- m + (e^g - 1) m, with e^g - 1 off by 2^-24 of |g|, or (past == false), beyond half a token's memory, m <- e^g m.  One number for e^g
// would be off by up to 2^-24 of itself, always the same way for a decay that does not change, so that a state which remembers n of about 1 / |g| tokens would be off
// by n times that (fp32 prompts of 2000 tokens 2.6e-5 of the state's norm; so 4e-7).  A strong decay has to leave nothing of what was before, which a sum with it would.
struct LaDecay {
    float by;
    bool past;
};
__device__ __forceinline__ LaDecay la_decay(float g)
{
    const bool past = fabsf(g) <= 0.6875f;
    return {past ? expm1f(g) : expf(g), past};
}

// A token for all warps of a CTA: y and x in fp32, the CTA's rows of cs z, and the decay.
template <int NV, int RT>
struct LaStaged {
    float4 y[8 * NV], x[8 * NV];
    float z[16 * RT];
    LaDecay a;
};

// A lane's share of one token as it arrives.
template <typename T, int NV, int RT>
struct LaToken {
    static constexpr int SHARE = (32 * NV + 127) / 128, ROWS = (16 * RT + 31) / 32;
    Pack<T, 4> x[SHARE], y[SHARE];
    T z[ROWS];
    float g;
};

// One CTA of W <= 4 warps: 4 RT W rows of one head's state.  RT: rows of a lane; NV: its float4 blocks of a row.
template <typename T, int NV, int RT, bool SEGMENTS>
__global__ void __launch_bounds__(128, RT * NV >= 16 ? 4 : RT * NV >= 8 ? 5 : 6) la_token_kernel(const LaRun A, int vec)
{
    __shared__ LaStaged<NV, RT> staged[2][4];  // W tokens, while the next W arrive
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5, cl = lane & 7, grp = lane >> 3;
    const int rows = 4 * RT * W;  // of the CTA
    const unsigned per_head = A.DV / rows, of_all = blockIdx.x / per_head, nh = SEGMENTS ? of_all / A.segments : of_all;
    const int first = (int)(blockIdx.x - of_all * per_head) * rows, segment = SEGMENTS ? (int)(of_all - nh * A.segments) : 0;
    const int n = nh / A.H, h = nh - n * A.H;

    begin_after();
    const LaSequence s = la_sequence(A, n);
    if (!s.ok) {
        if (threadIdx.x == 0) atomicOr(&g_la_token_status, 1);
        return;
    }
    // the walk's tokens of this CTA, and whether they are the last
    long long start = 0, end = s.hi - s.lo;
    bool is_last = true;
    if (SEGMENTS) {
        start = (long long)segment * A.per;
        if (segment > 0 && start >= end) return;
        if (start + A.per < end) {
            end = start + A.per;
            is_last = false;
        }
    }
    const long long len = end - start;
    const T *xh = (const T*)A.x + (h % A.xh) * A.xs1, *yh = (const T*)A.y + (h % A.yh) * A.ys1, *zh = (const T*)A.z + (h % A.zh) * A.zs1 + first;

    // token i of the walk
    LaToken<T, NV, RT> in;
    auto load = [&](long long i) {
        const long long row = A.reverse ? s.hi - 1 - start - i : s.lo + start + i;
        in.g = 0.f;
        if (!A.reverse || start + i > 0) in.g = ld_any(A.g, (row + A.reverse) * A.gs0 + h * A.gs1, A.gate_dtype);
#pragma unroll
        for (int b = 0; b < in.ROWS; ++b)
            if (32 * b + lane < rows) in.z[b] = ld_plain(zh + row * A.zs0 + 32 * b + lane);
#pragma unroll
        for (int b = 0; b < in.SHARE; ++b) {
            const int c = 128 * b + 4 * lane;
            if (c < A.DK) {
                in.y[b] = ld_pack<T, 4>(yh + row * A.ys0 + c, vec);
                in.x[b] = ld_pack<T, 4>(xh + row * A.xs0 + c, vec);
            }
        }
    };
    auto stage = [&](LaStaged<NV, RT>& S) {
#pragma unroll
        for (int b = 0; b < in.SHARE; ++b) {
            const int c = 128 * b + 4 * lane;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f), x = y;
            if (c < A.DK) {
                y = make_float4(in.y[b].get(0), in.y[b].get(1), in.y[b].get(2), in.y[b].get(3));
                x = make_float4(in.x[b].get(0), in.x[b].get(1), in.x[b].get(2), in.x[b].get(3));
            }
            if (c < 32 * NV) {
                S.y[c / 4] = y;
                S.x[c / 4] = x;
            }
        }
#pragma unroll
        for (int b = 0; b < in.ROWS; ++b)
            if (32 * b + lane < rows) S.z[32 * b + lane] = A.cs * to_f32(in.z[b]);
        if (lane == 0) S.a = la_decay(in.g);
    };
    if (warp < len) load(warp);

    // rows first + row_in + r of the state, r < RT
    const int row_in = warp * 4 * RT + grp * RT;
    const long long head = (long long)h * A.DV * A.DK;
    f2 m[RT][NV][2];
    {
        const float* from = A.s_in + s.in * A.in_stride + head;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int b = 0; b < NV; ++b) {
                const int c = 32 * b + 4 * cl, j = first + row_in + r;
                ulonglong2 v = make_ulonglong2(0, 0);
                if (SEGMENTS && (segment > 0 || !is_last)) {
                    const float* left = A.states + (long long)nh * A.segments * A.DK * A.DV;
                    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int k = segment > 0; k <= segment && c < A.DK; ++k) {
                        const float* d = left + (long long)k * A.DK * A.DV + c * A.DV + j;
                        const float a = k > 1 ? A.decays[nh * A.segments + k] : 0.f;
                        w.x = k > 1 ? fmaf(a, w.x, d[0]) : d[0];
                        w.y = k > 1 ? fmaf(a, w.y, d[A.DV]) : d[A.DV];
                        w.z = k > 1 ? fmaf(a, w.z, d[2 * A.DV]) : d[2 * A.DV];
                        w.w = k > 1 ? fmaf(a, w.w, d[3 * A.DV]) : d[3 * A.DV];
                    }
                    v = make_ulonglong2(pack2(w.x, w.y), pack2(w.z, w.w));
                } else if (s.in >= 0 && c < A.DK) {
                    if (!A.transposed_in) v = *reinterpret_cast<const ulonglong2*>(from + j * A.DK + c);
                    else
                        v = make_ulonglong2(pack2(from[c * A.DV + j], from[(c + 1) * A.DV + j]),
                                            pack2(from[(c + 2) * A.DV + j], from[(c + 3) * A.DV + j]));
                }
                m[r][b][0] = v.x;
                m[r][b][1] = v.y;
            }
    }

    // After the exchange between a row's 8 lanes, kShare of them hold the sum of row `mine` of the RT.
    constexpr int kShare = 8 / RT;
    const int mine = cl / kShare;
    const bool writes = (cl & (kShare - 1)) == 0;

    if (warp < len) stage(staged[0][warp]);
    if (W + warp < len) load(W + warp);
    const int shift = A.out_dtype == GDN_F32 ? 2 : 1;
    const long long step = (A.reverse ? -1ll : 1ll) * (((long long)A.H * A.DV) << shift);
    char* out = (char*)A.out + ((((A.reverse ? s.hi - 1 - start : s.lo + start) * A.H + h) * A.DV + first + row_in + mine) << shift);
    int set = 0;
    for (long long t0 = 0; t0 < len; t0 += W, set ^= 1) {
        __syncthreads();
        // the tokens after these W, staged by the warps while they are in them
        if (t0 + W + warp < len) {
            stage(staged[set ^ 1][warp]);
            if (t0 + 2 * W + warp < len) load(t0 + 2 * W + warp);
        }
        const int now = len - t0 < W ? (int)(len - t0) : W;
        for (int i = 0; i < now; ++i) {
            const LaStaged<NV, RT>& S = staged[set][i];
            const f2 aa = pack2(S.a.by, S.a.by);
            f2 zz[RT], o2[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const float z = S.z[row_in + r];
                zz[r] = pack2(z, z);
                o2[r] = 0;
            }
            auto update = [&](auto past) {
#pragma unroll
                for (int b = 0; b < NV; ++b) {
                    const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(&S.y[8 * b + cl]);
                    const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&S.x[8 * b + cl]);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        f2 &m0 = m[r][b][0], &m1 = m[r][b][1];
                        m0 = fma2(m0, aa, past.value ? fma2(y.x, zz[r], m0) : mul2(y.x, zz[r]));
                        m1 = fma2(m1, aa, past.value ? fma2(y.y, zz[r], m1) : mul2(y.y, zz[r]));
                        o2[r] = fma2(m0, x.x, o2[r]);
                        o2[r] = fma2(m1, x.y, o2[r]);
                    }
                }
            };
            if (S.a.past) update(std::true_type{});
            else update(std::false_type{});
            float o[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) o[r] = sum2(o2[r]);
            // reduce-scatter of the RT sums over the 8 lanes, then a butterfly over the lanes that share one
            int bit = 4;
#pragma unroll
            for (int n2 = RT / 2; n2 >= 1; n2 >>= 1, bit >>= 1) {
                const bool up = (cl & bit) != 0;
#pragma unroll
                for (int e = 0; e < n2; ++e) {
                    const float send = up ? o[e] : o[n2 + e], keep = up ? o[n2 + e] : o[e];
                    o[e] = keep + __shfl_xor_sync(kFull, send, bit);
                }
            }
#pragma unroll
            for (int b = kShare / 2; b >= 1; b >>= 1) o[0] += __shfl_xor_sync(kFull, o[0], b);
            if (writes) st_any(out, 0, A.out_dtype, A.co * o[0]);
            out += step;
        }
    }

    if (s.out < 0 || !is_last) return;
    float last = 1.f;  // backwards, the state before token 0
    if (A.reverse && s.hi > s.lo) last = expf(ld_any(A.g, s.lo * A.gs0 + h * A.gs1, A.gate_dtype));
    const f2 ll = pack2(last, last);
    float* to = A.s_out + s.out * A.out_stride + head;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int b = 0; b < NV; ++b) {
            const int c = 32 * b + 4 * cl, j = first + row_in + r;
            if (A.reverse) {
                m[r][b][0] = mul2(m[r][b][0], ll);
                m[r][b][1] = mul2(m[r][b][1], ll);
            }
            if (c < A.DK) {
                if (!A.transposed_out) *reinterpret_cast<ulonglong2*>(to + j * A.DK + c) = make_ulonglong2(m[r][b][0], m[r][b][1]);
                else {
                    const float2 lo = unpack2(m[r][b][0]), hi = unpack2(m[r][b][1]);
                    to[c * A.DV + j] = lo.x;
                    to[(c + 1) * A.DV + j] = lo.y;
                    to[(c + 2) * A.DV + j] = hi.x;
                    to[(c + 3) * A.DV + j] = hi.y;
                }
            }
        }
}

template <typename T, int NV, int RT>
int launch_g(const LaRun& A, int vec, cudaStream_t st)
{
    const int groups = A.DV / (4 * RT);  // warps' rows of a head
    int W = 4;
    while (groups % W != 0) --W;
    const long long ctas = (long long)A.n_seq * A.H * (groups / W);
    if constexpr (sizeof(T) == 2 && (NV == 2 || NV == 4)) {  // the chunked form's sizes
        if (A.segments) return launch_after(la_token_kernel<T, NV, RT, true>, (unsigned)(ctas * A.segments), 32 * W, 0, st, A, vec);
    }
    return launch_after(la_token_kernel<T, NV, RT, false>, (unsigned)ctas, 32 * W, 0, st, A, vec);
}

bool vec4(const void* ptr, long long s0, long long s1, size_t es) { return (uintptr_t)ptr % (4 * es) == 0 && s0 % 4 == 0 && s1 % 4 == 0; }

template <typename T>
int launch_t(const LaRun& A, cudaStream_t st)
{
    const int vec = vec4(A.x, A.xs0, A.xs1, sizeof(T)) && vec4(A.y, A.ys0, A.ys1, sizeof(T));
    // Few heads are spread over more warps of one row a lane; many take more rows a lane, so that a token's x and y
    // serve them all.  Rows of 128 columns in all, 24 tokens, 4 rows a lane against 1: 4096 rows 21 us and 19, 8192 21 and 23, 12288 25 and 25, 32768 33 and
    // 57; of 64 columns 8192 rows 20 and 19, 16384 22 and 23; of 256 (2 rows a lane) 4096 rows 27 and 27, 16384 38 and 62.
    const bool wide = (long long)A.n_seq * A.H * (A.segments ? A.segments : 1) * A.DV >= 16 * 4 * kNumSMs;
    if (A.DK <= 32) return wide ? launch_g<T, 1, 4>(A, vec, st) : launch_g<T, 1, 1>(A, vec, st);
    if (A.DK == 64) return wide ? launch_g<T, 2, 4>(A, vec, st) : launch_g<T, 2, 1>(A, vec, st);
    if (A.DK == 128) return wide ? launch_g<T, 4, 4>(A, vec, st) : launch_g<T, 4, 1>(A, vec, st);
    return wide ? launch_g<T, 8, 2>(A, vec, st) : launch_g<T, 8, 1>(A, vec, st);
}

}  // namespace

int launch_la_token(const LaRun& A, int dtype, cudaStream_t st)
{
    return dtype == GDN_F32 ? launch_t<float>(A, st) : dtype == GDN_BF16 ? launch_t<__nv_bfloat16>(A, st) : launch_t<__half>(A, st);
}

int la_token_take_status(void* stream, int* bad)
{
    const int e = la_read_words(&g_la_token_status, stream, 1, bad);
    return e || !*bad ? e : la_clear_word(&g_la_token_status, stream, 0);
}

}  // namespace gdn
