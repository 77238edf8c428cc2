// gdn_chain.h -- the pass over a sequence's 64-token chunks (gdn_internal.h has the formulas):
// one workgroup per (sequence, value head), one wave per 32 value columns.
//
// The columns of S are independent, so a wave keeps its K x 32 slice of S in fp32 registers for
// the whole sequence and needs nothing from the other waves: S, R and e leave one product in the
// very registers that are the next product's operand (C-layout tiles pairwise are a 16x16x32
// operand). The waves share what they read: K, Q, V rows and the chunk's record are copied to LDS
// (straight from memory, one chunk ahead), each once per workgroup, and read back as operands,
// K also transposed (ds_read_b64_tr_b16), so no operand is stored in a second layout. A 16-row
// operand read from LDS feeds two column tiles and the high and low parts: four products a read.
// The output product takes its operands in swapped roles, so a lane ends up with four
// consecutive columns of one token and stores eight bytes.
#pragma once

#include "gdn_internal.h"

namespace gdn {

// A wave's columns of the state (laid out as in forward_chain) to the workspace, [V][K] fp16.
template <int K>
__device__ __forceinline__ void keep_state(const f32x4 (&S)[K / 16][2], uint8_t *base, float *scale,
                                           int col0, int grp, int r)
{
    float m = 0.f;
#pragma unroll
    for (int t = 0; t < K / 16; ++t) m = max_abs(S[t][1], max_abs(S[t][0], m));
    const Scale f = scale_for(wave_max(m));
    const auto rs = kda::buffer_rsrc(base, 1u << 20);
#pragma unroll
    for (int t = 0; t < K / 16; ++t)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct)      // key dims 32 (t / 2) + 8 g + 4 (t % 2) .. + 3
            kda::bstore8<0>(rs, (col0 + 16 * ct + r) * K * 2 + 16 * grp, 64 * (t / 2) + 8 * (t % 2),
                            half4(S[t][ct], f.f));
    *scale = f.inv;
}

// A wave's columns of a [64 tokens][V] matrix in C-layout to the workspace, [V][64] fp16.
__device__ __forceinline__ void keep_rows(const f32x4 (&E)[4][2], uint8_t *base, float *scale,
                                          int col0, int grp, int r)
{
    float m = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t) m = max_abs(E[t][1], max_abs(E[t][0], m));
    const Scale f = scale_for(wave_max(m));
    const auto rs = kda::buffer_rsrc(base, 1u << 20);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct)
            kda::bstore8<0>(rs, (col0 + 16 * ct + r) * 128 + 8 * grp, 32 * t, half4(E[t][ct], f.f));
    *scale = f.inv;
}

// IN: planes of q and k, X: parts of the split operands; (1, 2) for bf16 io, (3, 3) for fp32 io
// OUT: the forward (o); else the backward's first pass (states and e kept, no q).
template <int K, int V, int IN, class R, bool OUT>
struct Stage {                              // LDS of one chunk
    static constexpr int MK = 64 * K * 2, MV = IN == 1 ? 64 * V * 2 : 0;    // fp32 v: from memory
    static constexpr int KM = 0, QM = IN * MK, VM = (OUT ? 2 : 1) * IN * MK;
    static constexpr int REC = VM + MV;
    static constexpr int KIB = OUT ? R::BYTES / 1024 : (R::RA + R::FR) / 1024;  // A and row scales
    static constexpr int BYTES = REC + KIB * 1024;
    static constexpr int BUFS = IN == 1 ? 2 : 1;        // fp32 io: three planes, one buffer
};

template <int K, int V, int IN, int X, class R, bool OUT>
__device__ __forceinline__ void forward_chain(const Params &p, int unit, uint8_t *lds,
                                              uint8_t *keep)
{
    using L = Stage<K, V, IN, R, OUT>;
    constexpr int NW = V / 32, NT = K / 16;
    static_assert(L::BYTES * L::BUFS <= 160 * 1024, "LDS of a compute unit");
    const int tid = threadIdx.x, lane = tid & 63, grp = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int s = unit / p.HV, j = unit % p.HV, h = j / p.G;
    const int64_t bos = kda::seq_bos(p.seq, s), eos = kda::seq_eos(p.seq, s, bos);
    const int nc = (int)((eos - bos + CT - 1) / CT);
    const size_t slot0 = (size_t)j * p.seq.n_slots + bos / CT + s;
    const uint8_t *const rec0 = p.rec + slot0 * R::BYTES;
    const int col0 = 32 * wave;

    auto stage = [&](int c, uint8_t *buf) {
        const int64_t t0 = bos + (int64_t)CT * c;
        const int nv = (int)(eos - t0 < CT ? eos - t0 : CT);
        const int64_t qk = (t0 * p.H + h) * K;
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            stage_rows<K, NW>(p.k[i] + qk, (int64_t)p.H * K, nv, buf + L::KM + i * L::MK, wave, lane);
            if constexpr (OUT) stage_rows<K, NW>(p.q[i] + qk, (int64_t)p.H * K, nv, buf + L::QM + i * L::MK, wave, lane);
        }
        if constexpr (IN == 1)
            stage_rows<V, NW>((const uint16_t *)p.v + (t0 * p.HV + j) * V, (int64_t)p.HV * V, nv,
                              buf + L::VM, wave, lane);
        stage_block<NW>(rec0 + (size_t)c * R::BYTES, L::KIB, buf + L::REC, wave, lane);
    };
    if (nc > 0) stage(0, lds);

    // row 4 g + i of state tile t is key dim 32 (t / 2) + 8 g + 4 (t % 2) + i: tiles 2s, 2s + 1
    // of a lane are then the eight consecutive key dims of a 16x16x32 operand
    f32x4 S[NT][2];
    const size_t st_off = ((size_t)s * p.HV + j) * K * V + col0 + r;
    auto state_at = [&](int t, int i, int ct) {
        return st_off + (size_t)(32 * (t / 2) + 8 * grp + 4 * (t % 2) + i) * V + 16 * ct;
    };
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[t][ct][i] = p.h0 ? p.h0[state_at(t, i, ct)] : 0.f;

#pragma unroll 1
    for (int c = 0; c < nc; ++c) {
        uint8_t *const buf = lds + (c % L::BUFS) * L::BYTES;
        const int64_t t0 = bos + (int64_t)CT * c;
        const int nv = (int)(eos - t0 < CT ? eos - t0 : CT);
        kda::vm_drain();                    // chunk c has arrived (all of this wave's loads)
        __syncthreads();
        if (L::BUFS == 2 && c + 1 < nc) stage(c + 1, lds + ((c + 1) % L::BUFS) * L::BYTES);
        const uint8_t *const rec = buf + L::REC;
        const float *const ra = (const float *)(rec + R::RA), *const rb = (const float *)(rec + R::RB);
        const float eg = *(const float *)(rec + R::EG);
        using KP = Keep<K, V>;
        uint8_t *const kept = OUT ? nullptr : keep + (slot0 + c) * KP::BYTES;
        float *const scales = (float *)(kept + KP::SCALE) + wave;
        if constexpr (!OUT) keep_state<K>(S, kept + KP::S, scales, col0, grp, r);
        f32x4 kS[4][2], O[4][2];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) kS[t][ct] = O[t][ct] = zero4();
        // K S and (Q S)^T
#pragma unroll
        for (int st = 0; st < K / 32; ++st) {
            Parts<X> sp[2];
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) sp[ct] = split<X>(S[2 * st][ct], S[2 * st + 1][ct]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int at = piece_at<K>(16 * t + r, 4 * st + grp);
                const Parts<IN> kk = lds_parts<IN>(buf + L::KM + at, L::MK);
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) kS[t][ct] = mm(kk, sp[ct], kS[t][ct]);
                if constexpr (OUT) {
                    const Parts<IN> qq = lds_parts<IN>(buf + L::QM + at, L::MK);
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) O[t][ct] = mm(sp[ct], qq, O[t][ct]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) S[t][ct] *= eg;
        // R = V - e^Gam (K S), as operands
        Parts<X> rp[2][2];
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            f32x4 x[2][2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = 2 * st + u;
                const f32x4 a = *(const f32x4 *)(ra + 16 * t + 4 * grp);
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) {
                    f32x4 v;
                    if constexpr (IN == 1) {
                        v = widen(lds_tr(buf + L::VM + piece_at<V>(16 * t + 4 * grp + (r >> 2),
                                                                   col0 / 8 + 2 * ct + ((r & 3) >> 1)) +
                                         8 * (r & 1)));
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = 16 * t + 4 * grp + i;
                            v[i] = ((const float *)p.v)[((t0 + (row < nv ? row : nv - 1)) * p.HV + j) * V +
                                                        col0 + 16 * ct + r];
                        }
                    }
                    x[u][ct] = v - a * kS[t][ct];
                }
            }
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) rp[st][ct] = split<X>(x[0][ct], x[1][ct]);
        }
        // e = A R
        f32x4 E[4][2];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            E[t][0] = E[t][1] = zero4();
#pragma unroll
            for (int st = 0; st <= t / 2; ++st) {
                const Parts<X> a = lds_parts<X>(rec + R::A + frag_index(t, st) * R::FR + lane * 16, R::MAT);
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) E[t][ct] = mm(a, rp[st][ct], E[t][ct]);
            }
        }
        if constexpr (OUT) {
            const float *const rc = (const float *)(rec + R::RC);
            // o = scale e^Gam (Q S) + M e
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float cs = rc[16 * t + r];
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) O[t][ct] *= cs;
            }
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                Parts<X> ep[2];
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) ep[ct] = split<X>(E[2 * st][ct], E[2 * st + 1][ct]);
#pragma unroll
                for (int t = 2 * st; t < 4; ++t) {
                    const Parts<X> m = lds_parts<X>(rec + R::M + frag_index(t, st) * R::FR + lane * 16, R::MAT);
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) O[t][ct] = mm(ep[ct], m, O[t][ct]);
                }
            }
            {
                constexpr int SZ = IN == 1 ? 2 : 4;
                // rows past the sequence end lie outside the resource: their stores are dropped
                const auto ob = kda::rows_in((uint8_t *)p.o + (t0 * p.HV + j) * (int64_t)V * SZ, nv,
                                             (int64_t)p.HV * V * SZ, V * SZ);
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct) {
                        const int at = ((16 * t + r) * p.HV * V + col0 + 16 * ct + 4 * grp) * SZ;
                        if constexpr (IN == 1)
                            kda::bstore8<0>(ob, at, 0, kda::to_bf16x4(O[t][ct]));
                        else
                            kda::bstore16<0>(ob, at, 0, O[t][ct]);
                    }
            }
        } else {
            keep_rows(E, kept + KP::E, scales + 2 * (V / 32), col0, grp, r);
        }
        // S += K^T (beta e^{gam - Gam} e)
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            Parts<X> dp[2];
            const f32x4 b0 = *(const f32x4 *)(rb + 32 * st + 4 * grp),
                        b1 = *(const f32x4 *)(rb + 32 * st + 16 + 4 * grp);
#pragma unroll
            for (int ct = 0; ct < 2; ++ct)
                dp[ct] = split<X>(b0 * E[2 * st][ct], b1 * E[2 * st + 1][ct]);
            const int row = 32 * st + 4 * grp + (r >> 2);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int piece = 4 * (t / 2) + (r & 3), half = 8 * (t % 2);
                const int at0 = piece_at<K>(row, piece) + half, at1 = piece_at<K>(row + 16, piece) + half;
                Parts<IN> kt;
#pragma unroll
                for (int i = 0; i < IN; ++i)
                    kt.p[i] = join(lds_tr(buf + L::KM + i * L::MK + at0), lds_tr(buf + L::KM + i * L::MK + at1));
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) S[t][ct] = mm(kt, dp[ct], S[t][ct]);
            }
        }
        if (L::BUFS == 1 && c + 1 < nc) {
            __syncthreads();                // every wave is done with the buffer
            stage(c + 1, lds);
        }
    }
    if (p.ht) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int ct = 0; ct < 2; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i) p.ht[state_at(t, i, ct)] = S[t][ct][i];
    }
}

}  // namespace gdn
