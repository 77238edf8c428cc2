// glr_backward.hip -- the gradients of the gated linear recurrence (include/glr.h). With dh_t the
// gradient of a loss with respect to h_t and m_t = e^{g_t} dh_t what token t hands to the one before it,
//     dh_t = dy_t + m_{t+1};   dx_t = beta_t dh_t;   dbeta_t = x_t dh_t;   dg_t = h_{t-1} m_t
// from m = dht behind the last token; dh0 = m_0. h_{t-1} is the forward's y_{t-1}. The same scan as the
// forward's, from the last token to the first: "token" below counts from the end.
//
// With y at hand no forward state is formed again: a pass over g, dy and y (with beta x and beta). Sums for A_log and dt_bias
// are fp32 over a lane's tokens of a step or tile (8 or 16, which its registers hold), fp64 over a sequence's steps and waves (a
// tile's waves), rounded to an fp32 row a sequence (a tile) and added in fp64 by a second launch of a workgroup for 64
// channels. bf16, us: 8 x 1000 tokens x 2048 channels 40 (4.1 TB/s), raw with the gate's gradients 70 (3.7 TB/s; vector
// instructions 57% of the SIMDs' time, with 1.6 waves on one: 512 workgroups' registers). 708 packed tokens x 512 channels fp32 raw:
// 13.5 + 3.9, two steps of the longest sequence and a launch.
#include "glr_scan.h"

namespace glr {

namespace {

template <typename T, int LPR, bool BETA>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(sizeof(T) == 2 ? 4 : 2))) void scan_back_kernel(BwdParams q)
{
    constexpr int VEC = 1, CH = LPR, R = 64 / LPR, STEP = R * K * W, E = sizeof(T);
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
    Gate gate[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) gate[v] = gate_of(p.pre, d + v);
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
    // offsets below zero).
    const uint32_t ds = (uint32_t)p.D * E;
    auto rows = [&](const void *base, int64_t stride, int64_t at, int64_t hi, int64_t beyond = 0) {
        return kda::rows_in((const T *)base + (bos + at) * stride + seq * beyond, (int)(hi - at), stride, p.D);
    };
    Raw<T, VEC> ng[K], nd[K];
    auto fetch = [&](int64_t s0) {
        const int64_t hi = n - s0, at = hi > STEP ? hi - STEP : 0;
        const auto gr = rows(p.g, p.gs, at, hi, p.ge), dr = rows(q.d_y, p.D, at, hi);
        const uint32_t row = (uint32_t)((int)(hi - at) - 1 - tok), gs = (uint32_t)p.gs * E;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            load(ng[k], gr, row * gs + d * E - k * gs);
            load(nd[k], dr, row * ds + d * E - k * ds);
        }
    };
    if (n > 0) fetch(0);
#pragma unroll
    for (int v = 0; v < VEC; ++v) asm volatile("" : : "v"(carry[v]));      // read before the first wave may write there
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
        for (int k = 0; k < K; ++k) load(cy[k], yr, (uint32_t)yrow * ds + d * E - k * ds);
        if constexpr (BETA) {
            const auto xr = rows(p.x, p.xs, at, hi, p.xe), br = rows(p.beta, p.bs, at, hi, p.be);
            const uint32_t xs = (uint32_t)p.xs * E, bs = (uint32_t)p.bs * E;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                load(cx[k], xr, (uint32_t)row * xs + d * E - k * xs);
                load(cb[k], br, (uint32_t)row * bs + d * E - k * bs);
            }
        }
        if (s0 + STEP < n) fetch(s0 + STEP);
        float c[K][VEC], act[K][VEC], G[VEC], end[VEC], m[VEC], least, most;
        log_decays<T>(cg, gate, p.pre.gate, row + 1, c, G, least, most);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) act[k][v] = c[k][v];
        const Form form = form_of<T>(least, most);
        uint32_t s = 0;
        by_form(form, [&](auto f) {
            constexpr Form F = decltype(f)::value;
            s = decays<T, F>(c);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                end[v] = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k) end[v] = apply<F>(c[k][v], s, k * VEC + v, end[v] + value(cd[k], v), 0.f);
            }
        });
        join<T, LPR, VEC>(G, end, carry, m, tot[buf], wave, lane);
        const auto dxr = rows(q.dx, p.D, at, hi), dgr = rows(q.dg, p.D, at, hi), dbr = rows(BETA ? q.dbeta : q.dx, p.D, at, hi);
        const uint32_t o0 = on ? (uint32_t)row * ds + d * E : PAST;
        float sA[VEC], sb[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) sA[v] = sb[v] = 0.f;
        by_kind(p.pre.gate, [&](auto kind) { by_form(form, [&](auto f) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float dx[VEC], dg[VEC], dbt[VEC];
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float dh = value(cd[k], v) + m[v];
                    m[v] = apply<decltype(f)::value>(c[k][v], s, k * VEC + v, dh, 0.f);
                    const float before = yrow - k == -1 && at == 0 ? first[v] : value(cy[k], v);
                    dx[v] = dh;
                    dg[v] = before * m[v];
                    if constexpr (BETA) {
                        const float b = value(cb[k], v);
                        const Sigmoid r = p.pre.beta_sigmoid ? sigmoid<T>(b) : Sigmoid{b, 1.f};
                        dx[v] *= r.s;
                        dbt[v] = value(cx[k], v) * dh * r.ds;
                    }
                    // (behind a sequence's end m is no token's gradient)
                    if (decltype(kind)::value != NONE)
                        dg[v] = gate[v].template back<T, decltype(kind)::value>(value(cg[k], v), act[k][v], k <= row ? dg[v] : 0.f, sA[v], sb[v]);
                }
                const uint32_t off = o0 - k * ds;
                store<T, VEC>(dx, dxr, off);
                store<T, VEC>(dg, dgr, off);
                if constexpr (BETA) store<T, VEC>(dbt, dbr, off);
            }
        }); });
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

// The sums of all rows of partial sums: 64 channels a workgroup, every sixteenth row a wave.
__global__ __launch_bounds__(1024) void params_kernel(const float *part_A, const float *part_b, int64_t rows, int D,
                                                      float *dA_log, float *ddt_bias)
{
    __shared__ double sums[2][16][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, d = blockIdx.x * 64 + lane;
    double a = 0.0, b = 0.0;
    if (d < D) {
#pragma unroll 4
        for (int64_t i = wave; i < rows; i += 16) {
            a += part_A[i * D + d];
            b += part_b[i * D + d];
        }
    }
    sums[0][wave][lane] = a;
    sums[1][wave][lane] = b;
    __syncthreads();
    if (wave > 1 || d >= D) return;
    double x = 0.0;
#pragma unroll
    for (int w = 0; w < 16; ++w) x += sums[wave][w][lane];
    if (wave == 0) dA_log[d] = (float)x;
    else if (ddt_bias) ddt_bias[d] = (float)x;
}

template <typename T, int LPR>
hipError_t launch(const BwdParams &q, hipStream_t st)
{
    const dim3 grid((unsigned)unit_grid(q.f.strips, q.f.seq.N, near_of(LPR * (int)sizeof(T))));
    if (q.f.beta)
        scan_back_kernel<T, LPR, true><<<grid, dim3(64 * W), 0, st>>>(q);
    else
        scan_back_kernel<T, LPR, false><<<grid, dim3(64 * W), 0, st>>>(q);
    return hipGetLastError();
}
template <typename T>
hipError_t launch_io(const BwdParams &q, int lanes, hipStream_t st)
{
    if (lanes == 64) return launch<T, 64>(q, st);
    if (lanes == 32) return launch<T, 32>(q, st);
    return lanes == 16 ? launch<T, 16>(q, st) : launch<T, 8>(q, st);
}

}  // namespace

hipError_t launch_bwd(const BwdParams &q, Shape s, hipStream_t st)
{
    return s.f32 ? launch_io<float>(q, s.lanes, st) : launch_io<uint16_t>(q, s.lanes, st);
}

hipError_t launch_params(const BwdParams &q, int64_t rows, float *dA_log, float *ddt_bias, hipStream_t st)
{
    params_kernel<<<dim3((q.f.D + 63) / 64), dim3(1024), 0, st>>>(q.part_A, q.part_b, rows, q.f.D, dA_log, ddt_bias);
    return hipGetLastError();
}

}  // namespace glr
