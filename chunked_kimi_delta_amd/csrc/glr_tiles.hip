// glr_tiles.hip -- the forward of the gated linear recurrence in tiles (glr_tiles.h). The
// mathematics is glr_forward.hip's.
//
// 131072 tokens x 2048 channels bf16: 375 us (4.3 TB/s, 83% of what a copy reaches; strips, 16 channels a workgroup, 943): each byte
// once (1.19 GB in, 0.57 out, words of the tiles among them), 3.6 waves on a SIMD, which wait 59% of their time, for inputs first
// and then for each other's words (about 2 us a tile). 21412 packed tokens x 4096 channels with raw gates 179 us: vector
// instructions fill 70% of the SIMDs' time (49 a value). A workgroup that fetched its next tile ahead of its hand-over
// took 550 us for the former: half the workgroups for its registers. Tiles of half the tokens 450, of words that wait
// for the window's before them (no spans) 480.
#include "glr_tiles.h"

namespace glr {

namespace {

__global__ __launch_bounds__(256) void clear_kernel(uint2 *p, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = make_uint2(0, 0);
}

constexpr int KT = 16, LPR = 64;        // tokens a lane, lanes a token
// Waves a workgroup: with beta registers leave room for five waves on a SIMD, which workgroups of four fill.
template <bool BETA> constexpr int waves() { return BETA ? 4 : 8; }
template <bool BETA> constexpr int tile_tokens() { return KT * waves<BETA>(); }

template <typename T, int VEC, bool BETA>
__global__ __launch_bounds__(64 * waves<BETA>()) void tile_kernel(Params p, Tiles x)
{
    constexpr int W = waves<BETA>(), CH = LPR * VEC, TILE = tile_tokens<BETA>(), E = sizeof(T);
    __shared__ Shared<CH, W> sh;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    // A strip does not stay on one XCD: 131072 tokens of 2048 channels took 497 us so, and 376 as here (with 2^n
    // channels its lines would lie in few of an L2's channels).
    const int strip = (blockIdx.x + blockIdx.x / (uint32_t)p.strips) % (uint32_t)p.strips;
    if (tid == 0) sh.number = atomicAdd(x.ticket + strip * TICKET, 1u);
    __syncthreads();
    int seq;
    int64_t t, bos, n;
    if (!tile_of(p.seq, TILE, __builtin_amdgcn_readfirstlane((int)sh.number), seq, t, bos, n)) return;
    const int ch = strip * CH + lane * VEC;
    const bool on = ch < p.D;
    const int d = on ? ch : 0, tok = wave * KT;
    const int64_t s0 = t * TILE;
    const int have = (int)(n - s0 < TILE ? n - s0 : TILE);
    const bool last = s0 + TILE >= n;
    float start[VEC], h[VEC], out[VEC];
    if (have > 0) {
        const uint32_t xs = (uint32_t)p.xs * E, gs = (uint32_t)p.gs * E, bs = (uint32_t)p.bs * E, ys = (uint32_t)p.D * E;
        auto rows = [&](const void *base, int64_t stride, int64_t beyond = 0) {
            return kda::rows_in((const T *)base + (bos + s0) * stride + seq * beyond, have, stride, p.D);
        };
        Raw<T, VEC> rg[KT], rx[KT], rb[BETA ? KT : 1];
        {
            const auto gr = rows(p.g, p.gs, p.ge), xr = rows(p.x, p.xs, p.xe);
            const uint32_t g0 = tok * gs + d * E, x0 = tok * xs + d * E;
#pragma unroll
            for (int k = 0; k < KT; ++k) load(rg[k], gr, g0 + k * gs);
#pragma unroll
            for (int k = 0; k < KT; ++k) load(rx[k], xr, x0 + k * xs);
            if constexpr (BETA) {
                const auto br = rows(p.beta, p.bs, p.be);
                const uint32_t b0 = tok * bs + d * E;
#pragma unroll
                for (int k = 0; k < KT; ++k) load(rb[k], br, b0 + k * bs);
            }
        }
        Gate gate[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            gate[v] = gate_of(p.pre, d + v);
            start[v] = t < SPAN && p.h0 && on ? p.h0[(int64_t)seq * p.D + d + v] : 0.f;
        }
        float c[KT][VEC], w[BETA ? KT : 1][VEC], G[VEC], end[VEC], least, most;
        log_decays<T>(rg, gate, p.pre.gate, have - tok, c, G, least, most);
        if constexpr (BETA) gated_inputs<T>(rx, rb, p.pre.beta_sigmoid, w);
        auto in = [&](int k, int v) {
            if constexpr (BETA) return w[k][v]; else return value(rx[k], v);
        };
        const Form form = form_of<T>(least, most);
        uint32_t s = 0;
        by_form(form, [&](auto f) {
            constexpr Form F = decltype(f)::value;
            s = decays<T, F>(c);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                end[v] = in(0, v);
#pragma unroll
                for (int k = 1; k < KT; ++k) end[v] = apply<F>(c[k][v], s, k * VEC + v, end[v], in(k, v));
            }
        });
        hand_over<T, LPR, VEC, W>(x, G, end, start, h, out, sh, bos / TILE + seq, seq, t, last, (int64_t)p.strips * CH, ch,
                                  wave, lane);
        const auto yr = rows(p.y, p.D);
        const uint32_t y0 = on ? tok * ys + d * E : PAST;    // channels past the last lie past every range
        by_form(form, [&](auto f) {
#pragma unroll
            for (int k = 0; k < KT; ++k) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) h[v] = apply<decltype(f)::value>(c[k][v], s, k * VEC + v, h[v], in(k, v));
                store<T, VEC>(h, yr, y0 + k * ys);
            }
        });
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) out[v] = p.h0 && on ? p.h0[(int64_t)seq * p.D + d + v] : 0.f;
    }
    if (last && p.ht && on && tid < LPR) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) p.ht[(int64_t)seq * p.D + d + v] = out[v];
    }
}

template <typename T, int VEC, bool BETA>
hipError_t launch(const Params &p, void *ws, hipStream_t st)
{
    const TilePlan r = plan_tiles(p, tile_tokens<BETA>(), LPR * VEC, ws);
    const hipError_t e = clear_tiles(r, st);
    if (e != hipSuccess) return e;
    tile_kernel<T, VEC, BETA><<<dim3((unsigned)(r.slots * p.strips)), dim3(64 * waves<BETA>()), 0, st>>>(p, r.x);
    return hipGetLastError();
}

}  // namespace

hipError_t clear_tiles(const TilePlan &r, hipStream_t st)
{
    const int64_t n = r.bytes / 8, blocks = (n + 255) / 256;
    clear_kernel<<<dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, st>>>((uint2 *)r.x.ticket, n);
    return hipGetLastError();
}

int64_t tiles_bytes(const Params &p, Shape s)
{
    return plan_tiles(p, p.beta ? tile_tokens<true>() : tile_tokens<false>(), LPR * s.vec, nullptr).bytes;
}

hipError_t launch_fwd_tiles(const Params &p, Shape s, void *ws, hipStream_t st)
{
    if (s.f32) return p.beta ? launch<float, 1, true>(p, ws, st) : launch<float, 1, false>(p, ws, st);
    if (p.beta) return launch<uint16_t, 1, true>(p, ws, st);
    return s.vec == 2 ? launch<uint16_t, 2, false>(p, ws, st) : launch<uint16_t, 1, false>(p, ws, st);
}

}  // namespace glr
