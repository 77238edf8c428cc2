// gdn_recurrent.hip -- the token recurrence of the gated delta rule, for serving steps and short
// dense batches:
//     S <- a S;   r = v - S^T k;   S <- S + beta k r^T;   o = scale S^T q       (a = e^g)
//
// One workgroup (4 waves) per (row, value head). A wave holds K / 4 rows of S, a lane two
// neighbouring columns (eight-byte loads and stores, a state row per 512 bytes), for all tokens
// of the call: the state is read and written once, which is what bounds a step. With one decay
// a token, both products of a token come from the state before it,
//     r = v - a (S^T k),   o = scale (a (S^T q) + (q.k) beta r),
// so the waves' partial sums meet once per token (in LDS, double buffered: one barrier).
// Measured: 64 rows (8 padding) of 32 heads, K = V = 128, 237 MB: 38.6 us where the states fit the last-level
// cache from step to step, 46 us (5.1 TB/s, what a copy reaches) where they do not. A call of 64 rows takes 42 us for
// one token, 47 for two, 60 for four, 86 for eight (states in the cache): 6 us a token more, its loads behind the
// barrier of the one before.
#include "gdn_internal.h"

namespace gdn {

namespace {

typedef __attribute__((ext_vector_type(2))) float f32x2;

__device__ __forceinline__ void put2(uint16_t *p, float x, float y) {
    const __bf16 a = (__bf16)x, b = (__bf16)y;
    *(uint32_t *)p = (uint32_t)__builtin_bit_cast(uint16_t, a) | (uint32_t)__builtin_bit_cast(uint16_t, b) << 16;
}
__device__ __forceinline__ void put2(float *p, float x, float y) { *(float2 *)p = make_float2(x, y); }

}  // namespace

template <int K, int V, typename T>
__global__ __launch_bounds__(256) void recurrent_kernel(StepParams p)
{
    constexpr int LPR = V / 2, RPI = 64 / LPR, NR = K / 4 / RPI;    // lanes a row, rows a load
    constexpr int KL = K / 64;
    __shared__ f32x2 kq[4][K];              // per wave: k, q of the token
    __shared__ f32x4 part[2][4][LPR];       // per wave and column pair: S^T k, S^T q
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int j = blockIdx.x, b = blockIdx.y, h = j / p.G;
    const int sub = lane / LPR, pair = lane % LPR;
    const T *const q = (const T *)p.q, *const k = (const T *)p.k, *const v = (const T *)p.v;
    const T *const g = (const T *)p.g, *const beta = (const T *)p.beta;
    T *const o = (T *)p.o;
    const int64_t tok0 = (int64_t)b * p.T;

    const int at = p.index ? p.index[b] : b;
    if (at < 0 || at >= p.slots) {          // padding: no state, o is zero
        for (int t = wave; t < p.T; t += 4)
            if (sub == 0) put2(o + ((tok0 + t) * p.HV + j) * V + 2 * pair, 0.f, 0.f);
        return;
    }
    const size_t st = ((size_t)at * p.HV + j) * K * V;
    const int row0 = wave * (K / 4) + sub;
    f32x2 S[NR];
    if (p.h0) {
#pragma unroll
        for (int i = 0; i < NR; ++i)
            S[i] = *(const f32x2 *)(p.h0 + st + (size_t)(row0 + RPI * i) * V + 2 * pair);
    } else {
#pragma unroll
        for (int i = 0; i < NR; ++i) S[i] = f32x2{0.f, 0.f};
    }
    for (int t = 0; t < p.T; ++t) {
        const int64_t tok = tok0 + t;
        float kv[KL], qv[KL], sk = 0.f, sq = 0.f, qk = 0.f;
#pragma unroll
        for (int u = 0; u < KL; ++u) {
            kv[u] = kda::to_f32(k[(tok * p.H + h) * K + lane + 64 * u]);
            qv[u] = kda::to_f32(q[(tok * p.H + h) * K + lane + 64 * u]);
            sk += kv[u] * kv[u];
            sq += qv[u] * qv[u];
            qk += qv[u] * kv[u];
        }
        float x = kda::to_f32(g[tok * p.HV + j]), bt = kda::to_f32(beta[tok * p.HV + j]);
        const float v0 = kda::to_f32(v[(tok * p.HV + j) * V + 2 * pair]),
                    v1 = kda::to_f32(v[(tok * p.HV + j) * V + 2 * pair + 1]);
        const float a = expf(activate_gate(p.pre, x, j));
        if (p.pre.beta_sigmoid) bt = exact_sigmoid(bt);
        qk = kda::wave_sum(qk);
        if (p.pre.qk_l2norm) {
            const float fk = 1.f / sqrtf(kda::wave_sum(sk) + kda::L2NORM_EPS),
                        fq = 1.f / sqrtf(kda::wave_sum(sq) + kda::L2NORM_EPS);
#pragma unroll
            for (int u = 0; u < KL; ++u) {
                kv[u] *= fk;
                qv[u] *= fq;
            }
            qk *= fk * fq;
        }
#pragma unroll
        for (int u = 0; u < KL; ++u) kq[wave][lane + 64 * u] = f32x2{kv[u], qv[u]};
        __builtin_amdgcn_wave_barrier();    // kq[wave] is this wave's own
        f32x4 acc = zero4();
        float kr[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const f32x2 e = kq[wave][row0 + RPI * i];
            kr[i] = e[0];
            acc[0] += S[i][0] * e[0];
            acc[1] += S[i][1] * e[0];
            acc[2] += S[i][0] * e[1];
            acc[3] += S[i][1] * e[1];
        }
        if constexpr (RPI == 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] += __shfl_xor(acc[e], 32);
        }
        if (sub == 0) part[t & 1][wave][pair] = acc;
        __syncthreads();
        f32x4 sum = part[t & 1][0][pair];
#pragma unroll
        for (int w = 1; w < 4; ++w) sum += part[t & 1][w][pair];
        const float r0 = bt * (v0 - a * sum[0]), r1 = bt * (v1 - a * sum[1]);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            S[i][0] = a * S[i][0] + kr[i] * r0;
            S[i][1] = a * S[i][1] + kr[i] * r1;
        }
        if (wave == (t & 3) && sub == 0)
            put2(o + (tok * p.HV + j) * V + 2 * pair, p.scale * (a * sum[2] + qk * r0),
                 p.scale * (a * sum[3] + qk * r1));
    }
    if (p.ht) {
#pragma unroll
        for (int i = 0; i < NR; ++i)
            *(float2 *)(p.ht + st + (size_t)(row0 + RPI * i) * V + 2 * pair) = make_float2(S[i][0], S[i][1]);
    }
}

template <int K, int V>
hipError_t launch_recurrent(const StepParams &p, bool f32, hipStream_t st)
{
    const dim3 grid(p.HV, p.B);
    if (f32)
        recurrent_kernel<K, V, float><<<grid, dim3(256), 0, st>>>(p);
    else
        recurrent_kernel<K, V, uint16_t><<<grid, dim3(256), 0, st>>>(p);
    return hipGetLastError();
}

#define GDN_INST(K, V) \
    template hipError_t launch_recurrent<K, V>(const StepParams &, bool, hipStream_t);
GDN_INST(64, 64)
GDN_INST(64, 128)
GDN_INST(128, 64)
GDN_INST(128, 128)
#undef GDN_INST

}  // namespace gdn
