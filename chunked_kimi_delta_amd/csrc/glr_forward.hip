// glr_forward.hip -- the forward of the gated linear recurrence and its serving step (include/glr.h):
//     h <- e^g h + beta x;   y = h
//
// The scan over strips (glr_scan.h). A value costs 6 to 15 instructions for its decay, a raw gate 14 and a sigmoid 5 more, and
// four of the scan's own, so bytes and instructions are of a size: 32 x 500 tokens x 2048 channels fp32 82 us (4.8 TB/s, 93% of
// what a copy reaches), 8 x 2048 x 4096 bf16 93 us (4.3 TB/s), raw 129 (4.2). Where strips are few it is a step's own time, 2.5 to 4 us
// for loads, the groups' scan, a barrier and the chain over the waves: 2048 x 2048 in 13 us. Kernel alone, 70 tokens of 256
// channels, raw: 5.2 us, two memory latencies.
//
// The step: a state is read and written once, by a thread of its own for all tokens of the call. 64 rows x 4096 channels 4.2 us
// (1 row x 2048 3.4): latency of index, state and inputs; the call takes 11.
#include "glr_scan.h"

namespace glr {

namespace {

template <typename T, int VEC, bool BETA>
struct Rows {
    Raw<T, VEC> x[K], g[K], b[BETA ? K : 1];
};

template <typename T, int LPR, bool BETA>
__global__ __launch_bounds__(64 * W) void scan_kernel(Params p)
{
    constexpr int VEC = 1, CH = LPR, R = 64 / LPR, STEP = R * K * W, E = sizeof(T);
    __shared__ Totals<CH> tot[2];
    int seq, strip;
    if (!unit_of(blockIdx.x, p.strips, p.seq.N, near_of(CH * E), seq, strip)) return;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int64_t bos = kda::seq_bos(p.seq, seq), n = kda::seq_eos(p.seq, seq, bos) - bos;
    const int ch = strip * CH + lane % LPR * VEC;
    const bool on = ch < p.D;
    const int d = on ? ch : 0, tok = (wave * R + lane / LPR) * K;
    Gate gate[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) gate[v] = gate_of(p.pre, d + v);
    float carry[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) carry[v] = p.h0 && on ? p.h0[(int64_t)seq * p.D + d + v] : 0.f;

    // offsets of this lane's first token in a step; a resource spans the step's rows
    const uint32_t xs = (uint32_t)p.xs * E, gs = (uint32_t)p.gs * E, bs = (uint32_t)p.bs * E, ys = (uint32_t)p.D * E;
    auto rows = [&](const void *base, int64_t stride, int64_t s0, int64_t beyond = 0) {
        const int64_t left = n - s0;
        return kda::rows_in((const T *)base + (bos + s0) * stride + seq * beyond, (int)(left < STEP ? left : STEP), stride, p.D);
    };
    Rows<T, VEC, BETA> next;
    auto fetch = [&](int64_t s0) {
        const auto xr = rows(p.x, p.xs, s0, p.xe), gr = rows(p.g, p.gs, s0, p.ge);
        const uint32_t g0 = tok * gs + d * E, x0 = tok * xs + d * E;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            load(next.g[k], gr, g0 + k * gs);
            load(next.x[k], xr, x0 + k * xs);
        }
        if constexpr (BETA) {
            const auto br = rows(p.beta, p.bs, s0, p.be);
            const uint32_t b0 = tok * bs + d * E;
#pragma unroll
            for (int k = 0; k < K; ++k) load(next.b[k], br, b0 + k * bs);
        }
    };
    if (n > 0) fetch(0);
#pragma unroll
    for (int v = 0; v < VEC; ++v) asm volatile("" : : "v"(carry[v]));      // read before the first wave may write there
    int buf = 0;
    for (int64_t s0 = 0; s0 < n; s0 += STEP, buf ^= 1) {
        const Rows<T, VEC, BETA> cur = next;
        if (s0 + STEP < n) fetch(s0 + STEP);
        float c[K][VEC], w[BETA ? K : 1][VEC], G[VEC], end[VEC], h[VEC], least, most;
        log_decays<T>(cur.g, gate, p.pre.gate, (int)(n - s0 < STEP ? n - s0 : STEP) - tok, c, G, least, most);
        if constexpr (BETA) gated_inputs<T>(cur.x, cur.b, p.pre.beta_sigmoid, w);
        auto in = [&](int k, int v) {
            if constexpr (BETA) return w[k][v]; else return value(cur.x[k], v);
        };
        const Form form = form_of<T>(least, most);
        uint32_t s = 0;
        auto local = [&](auto f) {
            constexpr Form F = decltype(f)::value;
            s = decays<T, F>(c);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                end[v] = in(0, v);
#pragma unroll
                for (int k = 1; k < K; ++k) end[v] = apply<F>(c[k][v], s, k * VEC + v, end[v], in(k, v));
            }
        };
        by_form(form, local);
        join<T, LPR, VEC>(G, end, carry, h, tot[buf], wave, lane);
        const auto yr = rows(p.y, p.D, s0);
        const uint32_t y0 = on ? tok * ys + d * E : PAST;    // channels past the last lie past every range
        by_form(form, [&](auto f) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) h[v] = apply<decltype(f)::value>(c[k][v], s, k * VEC + v, h[v], in(k, v));
                store<T, VEC>(h, yr, y0 + k * ys);
            }
        });
    }
    if (p.ht && on && tid < LPR) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) p.ht[(int64_t)seq * p.D + d + v] = carry[v];
    }
}

__device__ __forceinline__ void put(uint16_t *y, const float (&h)[1]) { *y = (uint16_t)bf16_bits(h[0]); }
__device__ __forceinline__ void put(uint16_t *y, const float (&h)[2]) { *(uint32_t *)y = bf16_bits(h[0], h[1]); }
__device__ __forceinline__ void put(float *y, const float (&h)[1]) { *y = h[0]; }
__device__ __forceinline__ void put(float *y, const float (&h)[2]) { *(float2 *)y = make_float2(h[0], h[1]); }

// A row's state on VEC channels a thread, its tokens one behind the other.
template <typename T, int VEC>
__global__ __launch_bounds__(256) void step_kernel(StepParams p)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = p.f.strips;
    if (i >= p.B * per) return;
    const int b = (int)(i / per), d = (int)(i % per) * VEC, D = p.f.D;
    const int at = p.index ? p.index[b] : b;
    const bool live = at >= 0 && at < p.slots;
    float h[VEC];
    Gate gate[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        h[v] = live ? p.state[(int64_t)at * D + d + v] : 0.f;
        gate[v] = gate_of(p.f.pre, d + v);
    }
    for (int t = 0; t < p.T; ++t) {
        const int64_t tok = (int64_t)b * p.T + t;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            if (live) {
                float g = kda::to_f32(((const T *)p.f.g)[tok * p.f.gs + b * p.f.ge + d + v]);
                by_kind(p.f.pre.gate, [&](auto n) { g = gate[v].template active<T, decltype(n)::value>(g); });
                float w = kda::to_f32(((const T *)p.f.x)[tok * p.f.xs + b * p.f.xe + d + v]), c, s;
                if (p.f.beta) {
                    const float x = kda::to_f32(((const T *)p.f.beta)[tok * p.f.bs + b * p.f.be + d + v]);
                    w *= p.f.pre.beta_sigmoid ? logistic<T>(x) : x;
                }
                decay<T>(g, c, s);
                h[v] = fmaf(c, h[v], fmaf(s, h[v], w));
            }
        }
        put((T *)p.f.y + tok * D + d, h);
    }
    if (live) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) p.state[(int64_t)at * D + d + v] = h[v];
    }
}

template <typename T, int LPR>
hipError_t launch(const Params &p, hipStream_t st)
{
    const dim3 grid((unsigned)unit_grid(p.strips, p.seq.N, near_of(LPR * (int)sizeof(T))));
    if (p.beta)
        scan_kernel<T, LPR, true><<<grid, dim3(64 * W), 0, st>>>(p);
    else
        scan_kernel<T, LPR, false><<<grid, dim3(64 * W), 0, st>>>(p);
    return hipGetLastError();
}
template <typename T>
hipError_t launch_io(const Params &p, int lanes, hipStream_t st)
{
    if (lanes == 64) return launch<T, 64>(p, st);
    if (lanes == 32) return launch<T, 32>(p, st);
    return lanes == 16 ? launch<T, 16>(p, st) : launch<T, 8>(p, st);
}

}  // namespace

hipError_t launch_fwd(const Params &p, Shape s, hipStream_t st)
{
    return s.f32 ? launch_io<float>(p, s.lanes, st) : launch_io<uint16_t>(p, s.lanes, st);
}

hipError_t launch_step(const StepParams &p, bool f32, int vec, hipStream_t st)
{
    const dim3 grid((unsigned)(((int64_t)p.B * p.f.strips + 255) / 256));
    if (f32 && vec == 2) step_kernel<float, 2><<<grid, dim3(256), 0, st>>>(p);
    else if (f32) step_kernel<float, 1><<<grid, dim3(256), 0, st>>>(p);
    else if (vec == 2) step_kernel<uint16_t, 2><<<grid, dim3(256), 0, st>>>(p);
    else step_kernel<uint16_t, 1><<<grid, dim3(256), 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace glr
