// glr_backward.hip -- the gradients of the gated linear recurrence (include/glr.h). With dh_t the
// gradient of a loss with respect to h_t and m_t = e^{g_t} dh_t what token t hands to the one before it,
//     dh_t = dy_t + m_{t+1};   dx_t = beta_t dh_t;   dbeta_t = x_t dh_t;   dg_t = h_{t-1} m_t
// from m = dht behind the last token; dh0 = m_0. h_{t-1} is the forward's y_{t-1}. The same scan as the
// forward's, from the last token to the first: "token" below counts from the end.
#include "glr_scan.h"

namespace glr {

namespace {

template <typename T, int VEC, int LPR, bool BETA>
__global__ __launch_bounds__(64 * W) void scan_back_kernel(BwdParams q)
{
    constexpr int CH = LPR * VEC, R = 64 / LPR, STEP = R * K * W, E = sizeof(T);
    __shared__ Totals<CH> tot[2];
    __shared__ double sums[2][W][CH];
    const Params &p = q.f;
    int seq, strip;
    if (!unit_of(blockIdx.x, p.strips, p.seq.N, near_of(CH * E), seq, strip)) return;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int64_t bos = kda::seq_bos(p.seq, seq), n = kda::seq_eos(p.seq, seq, bos) - bos;
    const int ch = strip * CH + lane % LPR * VEC;
    const bool on = ch < p.D, gated = p.pre.gate != 0;
    const int d = on ? ch : 0, tok = (wave * R + lane / LPR) * K;
    const Gate<T> gate0 = gate_of<T>(p.pre, d), gate1 = gate_of<T>(p.pre, VEC == 2 && on ? ch + 1 : d);
    float carry[VEC], first[VEC];           // m, and the state ahead of the first token
    double dA[VEC], db[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        carry[v] = q.dht && on ? q.dht[(int64_t)seq * p.D + d + v] : 0.f;
        first[v] = p.h0 && on ? p.h0[(int64_t)seq * p.D + d + v] : 0.f;
        dA[v] = db[v] = 0.0;
    }
    // A step takes the rows [max(lo, 0), hi) of the sequence, hi = n - s0 and lo = hi - STEP; token k of a
    // lane is row hi - 1 - tok - k, and rows before the sequence lie past every range (as unsigned
    // offsets).
    const uint32_t ds = (uint32_t)p.D * E;
    auto rows = [&](const void *base, int64_t stride, int64_t at, int64_t hi) {
        return kda::rows_in((const T *)base + (bos + at) * stride, (int)(hi - at), stride, p.D);
    };
    Raw<T, VEC> ng[K], nd[K];
    auto fetch = [&](int64_t s0) {
        const int64_t hi = n - s0, at = hi > STEP ? hi - STEP : 0;
        const auto gr = rows(p.g, p.gs, at, hi), dr = rows(q.d_y, p.D, at, hi);
        const int row = (int)(hi - at) - 1 - tok;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            load(ng[k], gr, row - k < 0 ? 0x80000000u : (uint32_t)(row - k) * (uint32_t)p.gs * E + d * E);
            load(nd[k], dr, row - k < 0 ? 0x80000000u : (uint32_t)(row - k) * ds + d * E);
        }
    };
    if (n > 0) fetch(0);
    int buf = 0;
    for (int64_t s0 = 0; s0 < n; s0 += STEP, buf ^= 1) {
        const int64_t hi = n - s0, at = hi > STEP ? hi - STEP : 0;
        const int row = (int)(hi - at) - 1 - tok;           // of this lane's token 0, from row `at`
        Raw<T, VEC> cg[K], cd[K], cy[K], cx[BETA ? K : 1], cb[BETA ? K : 1];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            cg[k] = ng[k];
            cd[k] = nd[k];
        }
        // y of the row before: a resource from row at - 1 on (from row 0 in the step that has it)
        const int64_t yat = at > 0 ? at - 1 : 0;
        const auto yr = rows(p.y, p.D, yat, hi);
        const int yrow = row - (at > 0 ? 0 : 1);
#pragma unroll
        for (int k = 0; k < K; ++k) load(cy[k], yr, yrow - k < 0 ? 0x80000000u : (uint32_t)(yrow - k) * ds + d * E);
        if constexpr (BETA) {
            const auto xr = rows(p.x, p.xs, at, hi), br = rows(p.beta, p.bs, at, hi);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                load(cx[k], xr, row - k < 0 ? 0x80000000u : (uint32_t)(row - k) * (uint32_t)p.xs * E + d * E);
                load(cb[k], br, row - k < 0 ? 0x80000000u : (uint32_t)(row - k) * (uint32_t)p.bs * E + d * E);
            }
        }
        if (s0 + STEP < n) fetch(s0 + STEP);
        float c[K][VEC], s[K][VEC], G[VEC], end[VEC], m[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const Gate<T> &gate = v ? gate1 : gate0;
            G[v] = end[v] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float g = gate.active(value(cg[k], v));
                if (gated && k > row) g = 0.f;
                decay<T>(g, c[k][v], s[k][v]);
                G[v] += g;
                const float u = end[v] + value(cd[k], v);
                end[v] = fmaf(c[k][v], u, s[k][v] * u);
            }
        }
        join<T, LPR, VEC>(G, end, carry, m, tot[buf], wave, lane);
        const auto dxr = rows(q.dx, p.D, at, hi), dgr = rows(q.dg, p.D, at, hi), dbr = rows(BETA ? q.dbeta : q.dx, p.D, at, hi);
        float sA[VEC], sb[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) sA[v] = sb[v] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float dx[VEC], dg[VEC], dbt[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const Gate<T> &gate = v ? gate1 : gate0;
                const float dh = value(cd[k], v) + m[v];
                m[v] = fmaf(c[k][v], dh, s[k][v] * dh);
                const float before = yrow - k == -1 && at == 0 ? first[v] : value(cy[k], v);
                dx[v] = dh;
                dg[v] = before * m[v];
                if constexpr (BETA) {
                    const float b = value(cb[k], v);
                    const Sigmoid r = p.pre.beta_sigmoid ? sigmoid<T>(b) : Sigmoid{b, 1.f};
                    dx[v] *= r.s;
                    dbt[v] = value(cx[k], v) * dh * r.ds;
                }
                if (gated) {
                    float a = 0.f, o = 0.f;
                    dg[v] = gate.back(value(cg[k], v), dg[v], a, o);
                    if (k <= row) {
                        sA[v] += a;
                        sb[v] += o;
                    }
                }
            }
            const uint32_t off = on && row - k >= 0 ? (uint32_t)(row - k) * ds + d * E : 0x80000000u;
            store<T, VEC>(dx, dxr, off);
            store<T, VEC>(dg, dgr, off);
            if constexpr (BETA) store<T, VEC>(dbt, dbr, off);
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            dA[v] += sA[v];
            db[v] += sb[v];
        }
    }
    if (q.dh0 && on && tid < LPR) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) q.dh0[(int64_t)seq * p.D + d + v] = carry[v];
    }
    if (gated) {                            // this sequence's sums over its tokens
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
#pragma unroll
            for (int m = LPR; m < 64; m *= 2) {
                dA[v] += __shfl_xor(dA[v], m);
                db[v] += __shfl_xor(db[v], m);
            }
            if (lane < LPR) {
                sums[0][wave][lane * VEC + v] = dA[v];
                sums[1][wave][lane * VEC + v] = db[v];
            }
        }
        __syncthreads();
        if (tid < 2 * CH && strip * CH + tid % CH < p.D) {
            double x = 0.0;
#pragma unroll
            for (int w = 0; w < W; ++w) x += sums[tid / CH][w][tid % CH];
            (tid < CH ? q.part_A : q.part_b)[(int64_t)seq * p.D + strip * CH + tid % CH] = (float)x;
        }
    }
}

// The sums of all sequences.
__global__ __launch_bounds__(256) void params_kernel(const float *part_A, const float *part_b, int N, int D,
                                                     float *dA_log, float *ddt_bias)
{
    const int d = blockIdx.x * 256 + threadIdx.x;
    if (d >= D) return;
    double a = 0.0, b = 0.0;
    for (int i = 0; i < N; ++i) {
        a += part_A[(int64_t)i * D + d];
        b += part_b[(int64_t)i * D + d];
    }
    dA_log[d] = (float)a;
    if (ddt_bias) ddt_bias[d] = (float)b;
}

template <typename T, int VEC, int LPR>
hipError_t launch(const BwdParams &q, hipStream_t st)
{
    const dim3 grid((unsigned)unit_grid(q.f.strips, q.f.seq.N, near_of(LPR * VEC * (int)sizeof(T))));
    if (q.f.beta)
        scan_back_kernel<T, VEC, LPR, true><<<grid, dim3(64 * W), 0, st>>>(q);
    else
        scan_back_kernel<T, VEC, LPR, false><<<grid, dim3(64 * W), 0, st>>>(q);
    return hipGetLastError();
}
template <typename T>
hipError_t launch_io(const BwdParams &q, Shape s, hipStream_t st)
{
    if (s.vec == 2) return s.lanes == 8 ? launch<T, 2, 8>(q, st) : launch<T, 2, 32>(q, st);
    return s.lanes == 8 ? launch<T, 1, 8>(q, st) : launch<T, 1, 32>(q, st);
}

}  // namespace

hipError_t launch_bwd(const BwdParams &q, Shape s, hipStream_t st)
{
    return s.f32 ? launch_io<float>(q, s, st) : launch_io<uint16_t>(q, s, st);
}

hipError_t launch_params(const BwdParams &q, float *dA_log, float *ddt_bias, hipStream_t st)
{
    params_kernel<<<dim3((q.f.D + 255) / 256), dim3(256), 0, st>>>(q.part_A, q.part_b, q.f.seq.N, q.f.D, dA_log, ddt_bias);
    return hipGetLastError();
}

}  // namespace glr
