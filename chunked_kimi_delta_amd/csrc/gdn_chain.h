// gdn_chain.h -- the pass over a sequence's 64-token chunks (gdn_internal.h has the formulas): one
// wave per 16 value columns of a (sequence, value head).
//
// The columns of S are independent, so a wave keeps its K x 16 slice of S in fp32 registers for
// the whole pass and needs nothing from the other waves: S, R and e leave one product in the very
// registers that are the next product's operand (C-layout tiles pairwise are a 16x16x32 operand).
// The waves of a workgroup (four or eight: 64 or 128 columns) share what they read: K, Q, V rows
// and the chunk's record are copied to LDS (straight from memory, one chunk ahead), each once, and
// read back as operands, K also transposed (ds_read_b64_tr_b16), so no operand is stored in a
// second layout. The output product takes its operands in swapped roles, so a lane ends up with
// four consecutive columns of one token and stores eight bytes.
#pragma once

#include "gdn_internal.h"

namespace gdn {

// What a pass over chunks is for.
enum Mode {
    OUT,        // the forward: o
    KEEP,       // the backward's first pass: states and e kept
    END,        // a segment's end state only
    PHI         // a segment's transition: its end state from the identity, without v
};

// IN: planes of q and k, X: parts of the split operands; (1, 2) for bf16 io, (3, 3) for fp32 io.
// C: columns of the workgroup.
template <int K, int C, int IN, class R, Mode M>
struct Stage {                              // LDS of one chunk
    static constexpr int MK = 64 * K * 2, MV = IN == 1 && M != PHI ? 64 * C * 2 : 0;   // fp32 v: from memory
    static constexpr int KM = 0, QM = IN * MK, VM = (M == OUT ? 2 : 1) * IN * MK;
    static constexpr int REC = VM + MV;
    static constexpr int KIB = M == OUT ? R::BYTES / 1024 : (R::RA + R::FR) / 1024;    // A, row scales
    static constexpr int BYTES = REC + KIB * 1024;
    static constexpr int BUFS = 2 * BYTES <= 160 * 1024 ? 2 : 1;
};

// A wave's slice of a K-row state: row 4 g + i of tile t is key dim 32 (t / 2) + 8 g + 4 (t % 2) + i,
// so that tiles 2s, 2s + 1 of a lane are the eight consecutive key dims of a 16x16x32 operand.
__device__ __forceinline__ int state_row(int t, int i, int grp) {
    return 32 * (t / 2) + 8 * grp + 4 * (t % 2) + i;
}

// The scales of what a pass keeps: every wave leaves the largest value of its columns in LDS before
// the barrier that each chunk has anyway, and behind it all take the largest of those. Two sets in
// turn, as a wave may be one barrier ahead.
template <int NW>
struct Maxima {
    float state[2][NW], rows[2][NW];
    static __device__ __forceinline__ Scale scale(const float (&m)[NW]) {
        float x = m[0];
#pragma unroll
        for (int w = 1; w < NW; ++w) x = __uint_as_float(max(__float_as_uint(x), __float_as_uint(m[w])));
        return scale_for(x);
    }
};

template <int N>
__device__ __forceinline__ float largest(const f32x4 (&x)[N]) {
    uint32_t m = 0;
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(x[t][i]) & 0x7fffffffu);   // NaN counts as the largest
    return wave_max(__uint_as_float(m));
}

// A wave's columns of the state to the workspace, [V][K] fp16 (column `col` of this lane).
template <int NT>
__device__ __forceinline__ void keep_state(const f32x4 (&S)[NT], Scale f, uint8_t *base, float *inv, int col,
                                           int grp)
{
    const auto rs = kda::buffer_rsrc(base, 1u << 20);
#pragma unroll
    for (int t = 0; t < NT; ++t)
        kda::bstore8<0>(rs, col * NT * 32 + 16 * grp, 64 * (t / 2) + 8 * (t % 2), half4(S[t], f.f));
    if (threadIdx.x == 0) *inv = f.inv;
}

// A wave's columns of a [64 tokens][V] matrix in C-layout to the workspace, [V][64] fp16.
__device__ __forceinline__ void keep_rows(const f32x4 (&E)[4], Scale f, uint8_t *base, float *inv, int col, int grp)
{
    const auto rs = kda::buffer_rsrc(base, 1u << 20);
#pragma unroll
    for (int t = 0; t < 4; ++t) kda::bstore8<0>(rs, col * 128 + 8 * grp, 32 * t, half4(E[t], f.f));
    if (threadIdx.x == 0) *inv = f.inv;
}

// The chunks [c0, c1) of one (sequence, value head) for the C columns from `cbase` of `ld` columns.
// init: the state's first element at c0 (row-major, `ld` columns), null for zeros (PHI: ignored);
// end: where to put the end state, or null.
template <int K, int V, int C, int IN, int X, class R, Mode M>
__device__ __forceinline__ void forward_chain(const Params &p, int s, int j, int c0, int c1, int cbase,
                                              const float *init, float *end, uint8_t *lds,
                                              uint8_t *keep = nullptr, Maxima<C / 16> *mx = nullptr)
{
    using L = Stage<K, C, IN, R, M>;
    static_assert(L::BYTES * L::BUFS <= 160 * 1024, "LDS of a compute unit");
    constexpr int NW = C / 16, NT = K / 16, LD = M == PHI ? K : V;
    const int tid = threadIdx.x, lane = tid & 63, grp = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = j / p.G;
    const int64_t bos = kda::seq_bos(p.seq, s), eos = kda::seq_eos(p.seq, s, bos);
    const size_t slot0 = (size_t)j * p.seq.n_slots + bos / CT + s;
    const int col0 = 16 * wave;             // within the workgroup's columns

    auto stage = [&](int c, uint8_t *buf) {
        const int64_t t0 = bos + (int64_t)CT * c;
        const int nv = (int)(eos - t0 < CT ? eos - t0 : CT);
        const int64_t qk = (t0 * p.H + h) * K;
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            stage_rows<K, NW>(p.k[i] + qk, (int64_t)p.H * K, nv, buf + L::KM + i * L::MK, wave, lane);
            if constexpr (M == OUT)
                stage_rows<K, NW>(p.q[i] + qk, (int64_t)p.H * K, nv, buf + L::QM + i * L::MK, wave, lane);
        }
        if constexpr (IN == 1 && M != PHI)
            stage_rows<C, NW>((const uint16_t *)p.v + (t0 * p.HV + j) * V + cbase, (int64_t)p.HV * V, nv,
                              buf + L::VM, wave, lane);
        stage_block<NW>(p.rec + (slot0 + c) * R::BYTES, L::KIB, buf + L::REC, wave, lane);
    };
    if (c0 < c1) stage(c0, lds);

    f32x4 S[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = state_row(t, i, grp), col = cbase + col0 + r;
            if constexpr (M == PHI)
                S[t][i] = row == col ? 1.f : 0.f;
            else
                S[t][i] = init ? init[(size_t)row * LD + col] : 0.f;
        }

    using KP = Keep<K, V>;
    auto kept = [&](int c) { return keep + (slot0 + c) * KP::BYTES; };
    f32x4 E[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) E[t] = zero4();
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
        uint8_t *const buf = lds + ((c - c0) % L::BUFS) * L::BYTES;
        const int64_t t0 = bos + (int64_t)CT * c;
        const int nv = (int)(eos - t0 < CT ? eos - t0 : CT);
        if constexpr (M == KEEP) {
            const float a = largest(S), b = largest(E);
            if (lane == 0) {
                mx->state[c & 1][wave] = a;
                mx->rows[c & 1][wave] = b;
            }
        }
        kda::vm_drain();                    // chunk c has arrived (all of this wave's copies)
        __syncthreads();
        if (L::BUFS == 2 && c + 1 < c1) stage(c + 1, lds + ((c + 1 - c0) % L::BUFS) * L::BYTES);
        if constexpr (M == KEEP) {          // S of this chunk, e of the one before
            float *const inv = (float *)(kept(c) + KP::SCALE);
            keep_state(S, mx->scale(mx->state[c & 1]), kept(c) + KP::S, inv, cbase + col0 + r, grp);
            if (c > c0)
                keep_rows(E, mx->scale(mx->rows[c & 1]), kept(c - 1) + KP::E, (float *)(kept(c - 1) + KP::SCALE) + 2,
                          cbase + col0 + r, grp);
        }
        const uint8_t *const rec = buf + L::REC;
        const float *const ra = (const float *)(rec + R::RA), *const rb = (const float *)(rec + R::RB);
        const float eg = *(const float *)(rec + R::EG);
        f32x4 kS[4], O[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) kS[t] = O[t] = zero4();
        // K S and (Q S)^T
#pragma unroll
        for (int st = 0; st < K / 32; ++st) {
            const Parts<X> sp = split<X>(S[2 * st], S[2 * st + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int at = piece_at<K>(16 * t + r, 4 * st + grp);
                kS[t] = mm(lds_parts<IN>(buf + L::KM + at, L::MK), sp, kS[t]);
                if constexpr (M == OUT) O[t] = mm(sp, lds_parts<IN>(buf + L::QM + at, L::MK), O[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) S[t] *= eg;
        // R = V - e^Gam (K S), as operands
        Parts<X> rp[2];
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            f32x4 x[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = 2 * st + u;
                const f32x4 a = *(const f32x4 *)(ra + 16 * t + 4 * grp);
                f32x4 v = zero4();
                if constexpr (M == PHI) {
                } else if constexpr (IN == 1) {
                    v = widen(lds_tr(buf + L::VM + piece_at<C>(16 * t + 4 * grp + (r >> 2),
                                                               col0 / 8 + ((r & 3) >> 1)) + 8 * (r & 1)));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 16 * t + 4 * grp + i;
                        v[i] = ((const float *)p.v)[((t0 + (row < nv ? row : nv - 1)) * p.HV + j) * V +
                                                    cbase + col0 + r];
                    }
                }
                x[u] = v - a * kS[t];
            }
            rp[st] = split<X>(x[0], x[1]);
        }
        // e = A R
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            E[t] = zero4();
#pragma unroll
            for (int st = 0; st <= t / 2; ++st)
                E[t] = mm(lds_parts<X>(rec + R::A + frag_index(t, st) * R::FR + lane * 16, R::MAT), rp[st], E[t]);
        }
        // S += K^T (beta e^{gam - Gam} e)
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const f32x4 b0 = *(const f32x4 *)(rb + 32 * st + 4 * grp),
                        b1 = *(const f32x4 *)(rb + 32 * st + 16 + 4 * grp);
            const Parts<X> dp = split<X>(b0 * E[2 * st], b1 * E[2 * st + 1]);
            const int row = 32 * st + 4 * grp + (r >> 2);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int piece = 4 * (t / 2) + (r & 3), half = 8 * (t % 2);
                const int at0 = piece_at<K>(row, piece) + half, at1 = piece_at<K>(row + 16, piece) + half;
                Parts<IN> kt;
#pragma unroll
                for (int i = 0; i < IN; ++i)
                    kt.p[i] = join(lds_tr(buf + L::KM + i * L::MK + at0), lds_tr(buf + L::KM + i * L::MK + at1));
                S[t] = mm(kt, dp, S[t]);
            }
        }
        if constexpr (M == OUT) {           // o = scale e^Gam (Q S) + M e
            const float *const rc = (const float *)(rec + R::RC);
#pragma unroll
            for (int t = 0; t < 4; ++t) O[t] *= rc[16 * t + r];
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                const Parts<X> ep = split<X>(E[2 * st], E[2 * st + 1]);
#pragma unroll
                for (int t = 2 * st; t < 4; ++t)
                    O[t] = mm(ep, lds_parts<X>(rec + R::M + frag_index(t, st) * R::FR + lane * 16, R::MAT), O[t]);
            }
            constexpr int SZ = IN == 1 ? 2 : 4;
            // rows past the sequence end lie outside the resource: their stores are dropped
            const auto ob = kda::rows_in((uint8_t *)p.o + (t0 * p.HV + j) * (int64_t)V * SZ, nv,
                                         (int64_t)p.HV * V * SZ, V * SZ);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int at = ((16 * t + r) * p.HV * V + cbase + col0 + 4 * grp) * SZ;
                if constexpr (IN == 1)
                    kda::bstore8<0>(ob, at, 0, kda::to_bf16x4(O[t]));
                else
                    kda::bstore16<0>(ob, at, 0, O[t]);
            }
        }
        if (L::BUFS == 1 && c + 1 < c1) {
            __syncthreads();                // every wave is done with the buffer
            stage(c + 1, lds);
        }
    }
    if constexpr (M == KEEP) {
        if (c0 < c1) {
            const float b = largest(E);
            if (lane == 0) mx->rows[c1 & 1][wave] = b;
            __syncthreads();
            keep_rows(E, mx->scale(mx->rows[c1 & 1]), kept(c1 - 1) + KP::E, (float *)(kept(c1 - 1) + KP::SCALE) + 2,
                      cbase + col0 + r, grp);
        }
    }
    if (end) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                end[(size_t)state_row(t, i, grp) * LD + cbase + col0 + r] = S[t][i];
    }
}

}  // namespace gdn
