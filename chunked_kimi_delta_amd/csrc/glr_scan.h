// glr_scan.h -- one workgroup's scan over a sequence's tokens for a strip of channels, in either
// direction of time.
//
// A wave has 64 / LPR groups of LPR lanes, a lane a channel and K tokens of each step (two channels a lane take the
// registers of a second workgroup on a compute unit: fp32 gradients of 8 x 1000 x 2048 179 us for 145): a
// step takes 64 / LPR x K x W tokens in order of (wave, group, token). A lane runs its tokens from a zero
// state; a scan over the groups and the waves' totals in LDS then give the state that it starts from, and
// it runs them again. The workgroup's own state goes from step to step in registers, and the next step's inputs are
// fetched ahead of the current one's work (behind it: 83 -> 86 us for 16384 x 1000): no workgroup waits for another.
#pragma once

#include <type_traits>

#include "glr_internal.h"

namespace glr {

// What a wave's tokens do to a state: h <- (c + s) h + E, for every channel of the strip.
template <int CH>
struct Totals {
    float c[W][CH], s[W][CH], E[W][CH];
};

// The values that the lower and the upper of each two neighbouring blocks of M lanes hold, in both.
template <int M>
__device__ __forceinline__ void both(float x, float &lo, float &up) {
    if constexpr (M == 8) {             // the halves of a row of 16 lanes: banks 0, 1 and 2, 3
        lo = __builtin_amdgcn_update_dpp(x, x, 0x118, 0xf, 0xc, false);     // row_shr:8
        up = __builtin_amdgcn_update_dpp(x, x, 0x108, 0xf, 0x3, false);     // row_shl:8
    } else {
        const uint32_t u = __builtin_bit_cast(uint32_t, x);
        const auto r = M == 16 ? __builtin_amdgcn_permlane16_swap(u, u, false, false)
                               : __builtin_amdgcn_permlane32_swap(u, u, false, false);
        lo = __builtin_bit_cast(float, (uint32_t)r[0]);
        up = __builtin_bit_cast(float, (uint32_t)r[1]);
    }
}

// A lane's tokens, and those of the groups before its own in its wave: h <- A h + E. G: sum of log decays.
struct Part {
    float A, E, G, A0, E0;
};
template <int M>
__device__ __forceinline__ void level(Part &p, int lane) {
    float al, au, el, eu, gl, gu;
    both<M>(p.A, al, au);
    both<M>(p.E, el, eu);
    both<M>(p.G, gl, gu);
    const bool upper = lane & M;
    p.E0 = fmaf(p.A0, upper ? el : 0.f, p.E0);
    p.A0 *= upper ? al : 1.f;
    p.E = fmaf(au, el, eu);
    p.A = al * au;
    p.G = gl + gu;
}

// From each lane's own tokens (sum G of log decays, end E of a zero state) to the state `in` that they
// start from; `carry`, the workgroup's state, moves behind the step's last token.
template <typename T, int LPR, int VEC>
__device__ __forceinline__ void join(const float (&G)[VEC], const float (&E)[VEC], float (&carry)[VEC],
                                     float (&in)[VEC], Totals<LPR * VEC> &tot, int wave, int lane) {
    const int at = lane % LPR;
    Part p[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        p[v] = Part{exp_<T>(G[v]), E[v], G[v], 1.f, 0.f};
        if constexpr (LPR <= 8) level<8>(p[v], lane);
        if constexpr (LPR <= 16) level<16>(p[v], lane);
        if constexpr (LPR <= 32) level<32>(p[v], lane);
    }
    if (lane < LPR) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float c, s;
            decay<T>(p[v].G, c, s);
            tot.c[wave][at * VEC + v] = c;
            tot.s[wave][at * VEC + v] = s;
            tot.E[wave][at * VEC + v] = p[v].E;
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        float h = carry[v], mine = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == wave) mine = h;
            h = fmaf(tot.c[w][at * VEC + v], h, fmaf(tot.s[w][at * VEC + v], h, tot.E[w][at * VEC + v]));
        }
        carry[v] = h;
        in[v] = fmaf(p[v].A0, mine, p[v].E0);
    }
}

// How a wave's decays of a step are held, by what they all are:
//   FAST   a alone, where rounding it to 24 bits costs at most 2^-17 of a state in all (bf16 io:
//          every |g| >= 2^-8; fp32 io, whose results would show that: every g < -1/2)
//   SLOW   e^g - 1 alone: every g in [-1/2, 0]
//   MIXED  (c, s)
// SLOW takes 6 instructions a decay and FAST the exponential's 5, with one or two a step; MIXED 15 and two.
enum Form { FAST, SLOW, MIXED };

template <typename T>
__device__ __forceinline__ Form form_of(float least, float most) {
    constexpr float FAST_MOST = sizeof(T) == 2 ? -0.00390625f : -0.5f;
    const bool fast = most <= FAST_MOST, slow = least >= -0.5f && most <= 0.f;
    if (__builtin_amdgcn_ballot_w64(!fast) == 0) return FAST;
    return __builtin_amdgcn_ballot_w64(!slow) == 0 ? SLOW : MIXED;
}

// A lane's decays of a step: c in place of the log decays, and a bit of s each.
template <typename T, Form F, int N, int VEC>
__device__ __forceinline__ uint32_t decays(float (&c)[N][VEC]) {
    static_assert(N * VEC <= 32, "a bit a decay");
    uint32_t s = 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float g = c[k][v];
            if (F == FAST) {
                c[k][v] = exp_<T>(g);
            } else if (F == SLOW) {
                c[k][v] = expm1_slow(g);
            } else {
                float one;
                decay<T>(g, c[k][v], one);
                s |= one != 0.f ? 1u << (k * VEC + v) : 0u;
                asm("" : "+v"(s));      // bit by bit: together they would take a register each
            }
        }
    return s;
}
template <class Fn>
__device__ __forceinline__ void by_form(Form f, Fn fn) {
    if (f == FAST) fn(std::integral_constant<Form, FAST>());
    else if (f == SLOW) fn(std::integral_constant<Form, SLOW>());
    else fn(std::integral_constant<Form, MIXED>());
}
// (s + c) h + w
template <Form F>
__device__ __forceinline__ float apply(float c, uint32_t s, int i, float h, float w) {
    if (F == FAST) return fmaf(c, h, w);
    if (F == SLOW) return fmaf(c, h, h + w);
    return fmaf(c, h, w + __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, h) & (uint32_t)((int32_t)(s << (31 - i)) >> 31)));
}

// Workgroup -> (sequence, strip). Workgroups go to the 8 XCDs in turn, and each XCD has its own L2:
// `near` neighbouring strips (those that share 128-byte lines) go to one XCD, one behind the other.
__device__ __forceinline__ bool unit_of(int wg, int strips, int N, int near, int &seq, int &strip) {
    const int groups = (strips + near - 1) / near, xcd = wg & 7, i = wg >> 3;
    const int64_t unit = (int64_t)(i / near) * 8 + xcd;
    seq = (int)(unit / groups);
    strip = (int)(unit % groups) * near + i % near;
    return seq < N && strip < strips;
}
inline int64_t unit_grid(int64_t strips, int64_t N, int near) {
    return ((strips + near - 1) / near * N + 7) / 8 * 8 * near;
}
// strips of `bytes` bytes a token that share a line
__host__ __device__ constexpr int near_of(int bytes) { return bytes >= 128 ? 1 : 128 / bytes; }

}  // namespace glr
