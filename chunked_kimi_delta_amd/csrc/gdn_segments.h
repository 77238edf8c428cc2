// gdn_segments.h -- the first pass over segments and the joining of their ends (Segments in
// gdn_internal.h).
#pragma once

#include "gdn_chain.h"

namespace gdn {

// E and PHI of the segments, 64 columns a workgroup: V / 64 workgroups for E, then K / 64 for PHI, per
// (slot, value head). E is not needed of a sequence's last segment, PHI neither of the first nor of the
// last. `part`: this workgroup's columns.
template <int K, int V, int IN, int X, class R>
__device__ __forceinline__ void forward_ends(const Params &p, int slot, int j, int part, uint8_t *lds)
{
    Segment g;
    if (!locate_segment(p.seq, p.seg.chunks, slot, &g) || g.last()) return;
    const size_t at = (size_t)slot * p.HV + j;
    if (part < V / 64) {
        const float *const h0 = p.h0 && g.i == 0 ? p.h0 + ((size_t)g.s * p.HV + j) * K * V : nullptr;
        if (h0) {                           // kept for the last pass
            float *const copy = p.seg.E + ((size_t)(slot + g.count - 1) * p.HV + j) * K * V;
            for (int i = threadIdx.x; i < K * 32; i += 256) {
                const int to = (i >> 5) * V + 64 * part + 2 * (i & 31);
                *(float2 *)(copy + to) = *(const float2 *)(h0 + to);
            }
        }
        forward_chain<K, V, 64, IN, X, R, END>(p, g.s, j, g.c0, g.c1, 64 * part, h0, p.seg.E + at * K * V, lds);
    } else if (g.i > 0) {
        forward_chain<K, V, 64, IN, X, R, PHI>(p, g.s, j, g.c0, g.c1, 64 * (part - V / 64), nullptr,
                                                  p.seg.PHI + at * 2 * K * K, lds);
    }
}

// The state that a segment starts from in the last pass.
template <int K, int V>
__device__ __forceinline__ const float *segment_start(const Params &p, const Segment &g, int slot, int j)
{
    const size_t kv = (size_t)K * V;
    if (g.i > 0) return p.seg.E + ((size_t)(slot - 1) * p.HV + j) * kv;
    if (!p.h0) return nullptr;
    return g.count == 1 ? p.h0 + ((size_t)g.s * p.HV + j) * kv
                        : p.seg.E + ((size_t)(slot + g.count - 1) * p.HV + j) * kv;
}

// LDS of a joining workgroup: per wave two buffers of its rows of PHI and of the segment's own end, and
// the running state as split operands.
template <int K, int X>
struct Join {
    static constexpr int ROWS = K / 4, PHI = ROWS * K * 4, BUF = PHI + ROWS * 64;
    static constexpr int SET = K / 32 * X * 1024, SETS = 8 * BUF, BYTES = SETS + SET;
};

// E_i <- PHI_i E_{i-1} + E_i for i = 1 .. count - 2, or (REV) G_i <- PHI_i^T G_{i+1} + G_i for
// i = count - 2 .. 1, of 16 columns of one (sequence, value head): four waves, K / 4 rows each. The
// running state is passed between the waves in LDS. What a step reads from memory
// takes far longer to arrive than the step, so each wave copies its own rows to LDS two segments ahead and
// waits by count for the older ones (loads into registers ahead of a loop made the compiler wait for all
// of them each time round: 3.4 us a segment, this way 2.1).
template <int K, int V, int X, bool REV>
__device__ __forceinline__ void join_ends(const Params &p, float *ends, int s, int j, int col0, uint8_t *lds)
{
    using L = Join<K, X>;
    constexpr int NS = K / 32, TW = K / 64, NP = K / 4;     // NP: 16-byte pieces of a row of PHI
    const int tid = threadIdx.x, lane = tid & 63, grp = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t bos = kda::seq_bos(p.seq, s), n = (kda::seq_eos(p.seq, s, bos) - bos + CT - 1) / CT;
    const int count = (int)((n + p.seg.chunks - 1) / p.seg.chunks);
    const int slot0 = (int)(bos / ((int64_t)CT * p.seg.chunks) + s);
    if (count < 3) return;
    auto end_of = [&](int i) { return ends + ((size_t)(slot0 + i) * p.HV + j) * K * V; };
    // step n = 0 .. count - 3 takes segment seg(n); before them segment seg(-1) is as it is
    auto seg = [&](int n) { return REV ? count - 2 - n : n + 1; };
    // row a of tile wave TW + u
    auto row_of = [&](int u, int a) { return state_row(wave * TW + u, a & 3, a >> 2); };
    uint8_t *const own = lds + wave * 2 * L::BUF;
    auto load = [&](int n, uint8_t *buf) {                  // COPIES copies
        const int i = seg(n < count - 3 ? n : count - 3);
        const float *const m = p.seg.PHI + (((size_t)(slot0 + i) * p.HV + j) * 2 + (REV ? 1 : 0)) * K * K;
#pragma unroll
        for (int q = 0; q < L::PHI / 1024; ++q) {
            const int at = q * 64 + lane, a = at / NP, piece = (at % NP) ^ (a & 15);
            copy16_to_lds(m, (uint32_t)(row_of(a >> 4, a & 15) * K * 4 + piece * 16), buf + q * 1024);
        }
#pragma unroll
        for (int u = 0; u < TW; ++u)
            copy16_to_lds(end_of(i) + col0, (uint32_t)(row_of(u, lane >> 2) * V * 4 + (lane & 3) * 16),
                          buf + L::PHI + u * 1024);
    };
    constexpr int COPIES = L::PHI / 1024 + TW, STORES = 4 * TW;
    auto share = [&](uint8_t *set, int u, f32x4 x) {        // this wave's tile as half an operand
        const int t = wave * TW + u;
#pragma unroll
        for (int k = 0; k < X; ++k) {
            const kda::bf16x4 y = kda::to_bf16x4(x);
            *(uint2 *)(set + ((t >> 1) * X + k) * 1024 + lane * 16 + (t & 1) * 8) = __builtin_bit_cast(uint2, y);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] -= (float)y[e];
        }
    };
#pragma unroll
    for (int u = 0; u < TW; ++u) {
        f32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = end_of(seg(-1))[(size_t)row_of(u, 4 * grp + e) * V + col0 + r];
        share(lds + L::SETS, u, x);
    }
    load(0, own);
    load(1, own + L::BUF);
#pragma unroll 1
    for (int n = 0; n < count - 2; ++n) {
        uint8_t *const buf = own + (n & 1) * L::BUF;
        // everything but the step before's stores and the next step's copies
        asm volatile("s_waitcnt vmcnt(%0)" :: "n"(COPIES + STORES) : "memory");
        if (n == 0) asm volatile("s_waitcnt vmcnt(%0)" :: "n"(COPIES) : "memory");
        Parts<X> a[TW][NS];
        f32x4 y[TW];
#pragma unroll
        for (int u = 0; u < TW; ++u) {
#pragma unroll
            for (int st = 0; st < NS; ++st) {
                const uint8_t *const row = buf + (16 * u + r) * K * 4;
                a[u][st] = split<X>(*(const f32x4 *)(row + ((8 * st + 2 * grp) ^ r) * 16),
                                    *(const f32x4 *)(row + ((8 * st + 2 * grp + 1) ^ r) * 16));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) y[u][e] = *(const float *)(buf + L::PHI + (16 * u + 4 * grp + e) * 64 + 4 * r);
        }
        kda::lds_barrier();
        const uint8_t *const from = lds + L::SETS;
#pragma unroll
        for (int st = 0; st < NS; ++st) {
            const Parts<X> b = lds_parts<X>(from + st * X * 1024 + lane * 16, 1024);
#pragma unroll
            for (int u = 0; u < TW; ++u) y[u] = mm(a[u][st], b, y[u]);
        }
        kda::lds_barrier();                                 // all waves have read the state
        const auto to = kda::buffer_rsrc(end_of(seg(n)), K * V * 4);
#pragma unroll
        for (int u = 0; u < TW; ++u) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y[u][e]), to,
                                                      (row_of(u, 4 * grp + e) * V + col0 + r) * 4, 0, 0);
            share(lds + L::SETS, u, y[u]);
        }
        load(n + 2, buf);                                   // (its reads are done: they went into a and y)
    }
    kda::vm_drain();                                        // no copy outlives its LDS
}

// Workgroups go to the eight XCDs in turn, each with its own L2: the `parts` workgroups of one unit get
// numbers eight apart, so that what they share is read into one L2 once. Grid: grid_for(units, parts).
__device__ __forceinline__ bool unit_of(int wg, int parts, int units, int *unit, int *part) {
    return kda::state_unit(wg, parts, units, unit, part);
}
inline unsigned grid_for(int64_t units, int parts) { return (unsigned)((units + 7) / 8 * 8 * parts); }

}  // namespace gdn
