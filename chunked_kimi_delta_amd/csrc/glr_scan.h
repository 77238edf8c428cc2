// glr_scan.h -- one workgroup's scan over a sequence's tokens for a strip of channels, in either
// direction of time.
//
// A wave has 64 / LPR groups of LPR lanes, a lane VEC neighbouring channels and K tokens of each step: a
// step takes 64 / LPR x K x W tokens in order of (wave, group, token). A lane runs its tokens from a zero
// state; a scan over the groups and the waves' totals in LDS then give the state that it starts from, and
// it runs them again. The workgroup's own state goes from step to step in registers: no workgroup waits
// for another.
#pragma once

#include "glr_internal.h"

namespace glr {

// What a wave's tokens do to a state: h <- (c + s) h + E, for every channel of the strip.
template <int CH>
struct Totals {
    float c[W][CH], s[W][CH], E[W][CH];
};

// From each lane's own tokens (sum G of log decays, end E of a zero state) to the state `in` that they
// start from; `carry`, the workgroup's state, moves behind the step's last token.
template <typename T, int LPR, int VEC>
__device__ __forceinline__ void join(const float (&G)[VEC], const float (&E)[VEC], float (&carry)[VEC],
                                     float (&in)[VEC], Totals<LPR * VEC> &tot, int wave, int lane) {
    const int at = lane % LPR;
    float A[VEC], e[VEC], g[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        g[v] = G[v];
        e[v] = E[v];
        A[v] = exp_<T>(G[v]);
    }
#pragma unroll
    for (int m = LPR; m < 64; m *= 2) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float a0 = __shfl_up(A[v], m), e0 = __shfl_up(e[v], m), g0 = __shfl_up(g[v], m);
            if (lane >= m) {
                e[v] = fmaf(A[v], e0, e[v]);
                A[v] *= a0;
                g[v] += g0;
            }
        }
    }
    if (lane >= 64 - LPR) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float c, s;
            decay<T>(g[v], c, s);
            tot.c[wave][at * VEC + v] = c;
            tot.s[wave][at * VEC + v] = s;
            tot.E[wave][at * VEC + v] = e[v];
        }
    }
    // the groups before this one
    float A0[VEC], e0[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        A0[v] = 1.f;
        e0[v] = 0.f;
        if constexpr (LPR < 64) {
            const float a = __shfl_up(A[v], LPR), x = __shfl_up(e[v], LPR);
            if (lane >= LPR) {
                A0[v] = a;
                e0[v] = x;
            }
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
        in[v] = fmaf(A0[v], mine, e0[v]);
    }
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
