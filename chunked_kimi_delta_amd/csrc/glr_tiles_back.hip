// glr_tiles_back.hip -- the gradients of the gated linear recurrence in tiles (glr_tiles.h): glr_backward.hip's
// mathematics, tiles and tokens counted from a sequence's end.
//
// 4 x 8192 tokens x 4096 channels bf16 284 us (4.7 TB/s, 91% of what a copy reaches), 4096 x 2048 22 + 2 us for the cleared words
// (84 MB: two rounds of tiles, whose first loads and last stores overlap with nothing), fp32 8192 x 2048 71 us (4.7 TB/s).
#include "glr_tiles.h"

namespace glr {

namespace {

constexpr int W = 8, LPR = 64;          // waves a workgroup, lanes a token
// Tokens a lane: with beta 16 would take more registers than two workgroups on a compute unit have.
template <bool BETA> constexpr int tokens() { return BETA ? 8 : 16; }
template <bool BETA> constexpr int tile_tokens() { return tokens<BETA>() * W; }

template <typename T, int VEC, bool BETA>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(4))) void tile_back_kernel(BwdParams q, Tiles x)
{
    constexpr int KB = tokens<BETA>(), TILE = tile_tokens<BETA>(), CH = LPR * VEC, E = sizeof(T);
    __shared__ Shared<CH, W> sh;
    const Params &p = q.f;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int strip = (blockIdx.x + blockIdx.x / (uint32_t)p.strips) % (uint32_t)p.strips;
    if (tid == 0) sh.number = atomicAdd(x.ticket + strip * TICKET, 1u);
    __syncthreads();
    const int slot = __builtin_amdgcn_readfirstlane((int)sh.number);
    int seq;
    int64_t t, bos, n;
    const bool there = tile_of(p.seq, TILE, slot, seq, t, bos, n);
    const int ch = strip * CH + lane * VEC;
    const bool on = ch < p.D, gated = p.pre.gate != 0;
    const int d = on ? ch : 0, tok = wave * KB;
    if (!there || n == 0) {
        if (gated && wave == 0 && on) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) q.part_A[(int64_t)slot * p.D + d + v] = q.part_b[(int64_t)slot * p.D + d + v] = 0.f;
        }
        if (there && q.dh0 && on && wave == 0) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) q.dh0[(int64_t)seq * p.D + d + v] = q.dht ? q.dht[(int64_t)seq * p.D + d + v] : 0.f;
        }
        return;
    }
    const int64_t s0 = t * TILE, hi = n - s0, at = hi > TILE ? hi - TILE : 0;   // rows [at, hi) of the sequence
    const bool last = hi <= TILE;                                               // (that is, its first token's tile)
    const int row = (int)(hi - at) - 1 - tok;                                   // of this lane's token 0, from row `at`
    const uint32_t ds = (uint32_t)p.D * E;
    auto rows = [&](const void *base, int64_t stride, int64_t from, int64_t beyond = 0) {
        return kda::rows_in((const T *)base + (bos + from) * stride + seq * beyond, (int)(hi - from), stride, p.D);
    };
    // rows before the sequence lie past every range, as unsigned offsets below zero
    auto fetch = [&](Raw<T, VEC> (&r)[KB], __amdgpu_buffer_rsrc_t b, int first, uint32_t stride) {
        const uint32_t o = (uint32_t)first * stride + d * E;
#pragma unroll
        for (int k = 0; k < KB; ++k) load(r[k], b, o - k * stride);
    };
    Raw<T, VEC> rg[KB], rd[KB], ry[KB], rx[BETA ? KB : 1], rb[BETA ? KB : 1];
    fetch(rg, rows(p.g, p.gs, at, p.ge), row, (uint32_t)p.gs * E);
    fetch(rd, rows(q.d_y, p.D, at), row, ds);
    // y of the row before: from row at - 1 on (from row 0 in the tile that has it)
    const int64_t yat = at > 0 ? at - 1 : 0;
    const int yrow = row - (at > 0 ? 0 : 1);
    fetch(ry, rows(p.y, p.D, yat), yrow, ds);
    if constexpr (BETA) {
        fetch(rx, rows(p.x, p.xs, at, p.xe), row, (uint32_t)p.xs * E);
        fetch(rb, rows(p.beta, p.bs, at, p.be), row, (uint32_t)p.bs * E);
    }
    Gate gate[VEC];
    float start[VEC], first[VEC], m[VEC], out[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        gate[v] = gate_of(p.pre, d + v);
        start[v] = t < SPAN && q.dht && on ? q.dht[(int64_t)seq * p.D + d + v] : 0.f;
        first[v] = last && p.h0 && on ? p.h0[(int64_t)seq * p.D + d + v] : 0.f;
    }
    float c[KB][VEC], act[KB][VEC], G[VEC], end[VEC], least, most;
    log_decays<T>(rg, gate, p.pre.gate, row + 1, c, G, least, most);
#pragma unroll
    for (int k = 0; k < KB; ++k)
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
            for (int k = 0; k < KB; ++k) end[v] = apply<F>(c[k][v], s, k * VEC + v, end[v] + value(rd[k], v), 0.f);
        }
    });
    hand_over<T, LPR, VEC, W>(x, G, end, start, m, out, sh, bos / TILE + seq, seq, t, last, (int64_t)p.strips * CH, ch, wave, lane);
    const auto dxr = rows(q.dx, p.D, at), dgr = rows(q.dg, p.D, at), dbr = rows(BETA ? q.dbeta : q.dx, p.D, at);
    const uint32_t o0 = on ? (uint32_t)row * ds + d * E : PAST;
    float sA[VEC], sb[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) sA[v] = sb[v] = 0.f;
    by_kind(p.pre.gate, [&](auto kind) { by_form(form, [&](auto f) {
#pragma unroll
        for (int k = 0; k < KB; ++k) {
            float dx[VEC], dg[VEC], dbt[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float dh = value(rd[k], v) + m[v];
                m[v] = apply<decltype(f)::value>(c[k][v], s, k * VEC + v, dh, 0.f);
                const float before = last && yrow - k == -1 ? first[v] : value(ry[k], v);
                dx[v] = dh;
                dg[v] = before * m[v];
                if constexpr (BETA) {
                    const float b = value(rb[k], v);
                    const Sigmoid r = p.pre.beta_sigmoid ? sigmoid<T>(b) : Sigmoid{b, 1.f};
                    dx[v] *= r.s;
                    dbt[v] = value(rx[k], v) * dh * r.ds;
                }
                // (ahead of the sequence's first row m is no token's gradient)
                if (decltype(kind)::value != NONE)
                    dg[v] = gate[v].template back<T, decltype(kind)::value>(value(rg[k], v), act[k][v], k <= row ? dg[v] : 0.f, sA[v], sb[v]);
            }
            const uint32_t off = o0 - k * ds;
            store<T, VEC>(dx, dxr, off);
            store<T, VEC>(dg, dgr, off);
            if constexpr (BETA) store<T, VEC>(dbt, dbr, off);
        }
    }); });
    if (last && q.dh0 && on && wave == 0) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) q.dh0[(int64_t)seq * p.D + d + v] = out[v];
    }
    if (gated) {                            // this tile's sums over its tokens: fp64 over the waves
        __syncthreads();                    // the maps' LDS is read
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            sh.c[wave][lane * VEC + v] = sA[v];
            sh.s[wave][lane * VEC + v] = sb[v];
        }
        __syncthreads();
        if (tid < 2 * CH && strip * CH + tid % CH < p.D) {
            double sum = 0.0;
#pragma unroll
            for (int w = 0; w < W; ++w) sum += tid < CH ? sh.c[w][tid % CH] : sh.s[w][tid % CH];
            (tid < CH ? q.part_A : q.part_b)[(int64_t)slot * p.D + strip * CH + tid % CH] = (float)sum;
        }
    }
}

template <typename T, int VEC, bool BETA>
hipError_t launch(const BwdParams &q, void *ws, hipStream_t st)
{
    const TilePlan r = plan_tiles(q.f, tile_tokens<BETA>(), LPR * VEC, ws);
    const hipError_t e = clear_tiles(r, st);
    if (e != hipSuccess) return e;
    tile_back_kernel<T, VEC, BETA><<<dim3((unsigned)(r.slots * q.f.strips)), dim3(64 * W), 0, st>>>(q, r.x);
    return hipGetLastError();
}

int tile_of(const Params &p) { return p.beta ? tile_tokens<true>() : tile_tokens<false>(); }

}  // namespace

int64_t tiles_back_bytes(const Params &p, Shape s) { return plan_tiles(p, tile_of(p), LPR * s.vec, nullptr).bytes; }
int64_t tiles_back_rows(const Params &p) { return p.seq.T_total / tile_of(p) + p.seq.N; }

hipError_t launch_bwd_tiles(const BwdParams &q, Shape s, void *ws, hipStream_t st)
{
    if (s.f32) return q.f.beta ? launch<float, 1, true>(q, ws, st) : launch<float, 1, false>(q, ws, st);
    if (!q.f.beta) return launch<uint16_t, 1, false>(q, ws, st);
    return s.vec == 2 ? launch<uint16_t, 2, true>(q, ws, st) : launch<uint16_t, 1, true>(q, ws, st);
}

}  // namespace glr
