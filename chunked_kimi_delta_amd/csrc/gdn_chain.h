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
//
// What bounds it: a chunk is a chain of dependent products and splits, 3.2 us for 64 columns alone (K = 128,
// bf16 io) and 3.5 with every compute unit busy (8.3 thousand clocks). By the counters the matrix core works 2.1
// thousand of those, LDS 2.2 (290 KB of K, Q and the record; 37% of it bank conflicts) and the vector
// instructions 2.2, each in turn. Reading operands a phase ahead took 16 heads x 4096 tokens
// without segments from 205 to 196 us; interleaving the two kinds of instructions by hand 209.
#pragma once

#include <type_traits>

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

// The scales of what a pass keeps: every wave leaves the largest value of its columns (of a state, and of each
// token of e or dR) in LDS before the barrier that each chunk has anyway, and behind it all take the largest
// of those. Two sets in turn, as a wave may be one barrier ahead.
template <int NW>
struct Maxima {
    float state[2][NW], rows[2][NW][64];
    static __device__ __forceinline__ Scale scale(const float (&m)[NW]) {
        uint32_t x = __float_as_uint(m[0]);
#pragma unroll
        for (int w = 1; w < NW; ++w) x = max(x, __float_as_uint(m[w]));
        return scale_for(__uint_as_float(x));
    }
};

template <int N>
__device__ __forceinline__ float largest(const f32x4 (&x)[N]) {
    uint32_t m = 0;
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(x[t][i]) & 0x7fffffffu);     // NaN counts
    return wave_max(__uint_as_float(m));
}

// The token whose maximum and scale a lane holds: those of element i of tile t are in lane 4 t + i of the 16
// that share its tokens.
__device__ __forceinline__ int scale_token(int grp, int r) { return 16 * (r >> 2) + 4 * grp + (r & 3); }

// The largest magnitude of each token over the wave's 16 columns, in scale_token order: halves of the 16 values
// are exchanged between lanes of a 16-lane row, then quarters, and so on.
__device__ __forceinline__ float largest_of_tokens(const f32x4 (&x)[4], int r)
{
    uint32_t v[16];
#pragma unroll
    for (int n = 0; n < 16; ++n) v[n] = __float_as_uint(x[n / 4][n % 4]) & 0x7fffffffu;    // NaN counts
    auto halve = [&](int bit, auto exchange) {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            if (n >= bit) break;
            const uint32_t keep = r & bit ? v[n + bit] : v[n], send = r & bit ? v[n] : v[n + bit];
            v[n] = max(keep, exchange(send));
        }
    };
    halve(8, [](uint32_t y) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)y, 0x128, 0xf, 0xf, false); });  // row_ror:8
    halve(4, [](uint32_t y) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)y, 0x141, 0xf, 0xf, false); });  // row_half_mirror
    halve(2, [](uint32_t y) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)y, 0x4e, 0xf, 0xf, false); });   // quad_perm 2,3,0,1
    halve(1, [](uint32_t y) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)y, 0xb1, 0xf, 0xf, false); });   // quad_perm 1,0,3,2
    return __uint_as_float(v[0]);
}

// A wave's columns of the state, or of a [64 tokens][V] matrix in C-layout, to the workspace (`col`: this
// lane's column).
template <class KP, int NT>
__device__ __forceinline__ void keep_state(const f32x4 (&S)[NT], Scale f, uint8_t *base, float *inv, int col,
                                           int grp)
{
    const auto rs = kda::buffer_rsrc(base, KP::BYTES);
#pragma unroll
    for (int t = 0; t < NT; ++t)
        kda::bstore8<0>(rs, KP::state_at(col, state_row(t, 0, grp)), 0, half4(S[t], f.f));
    if (threadIdx.x == 0) *inv = f.inv;
}

// Each token has a scale of its own: betas, values or gradients of o of the tokens of a chunk may differ by any
// factor, and so may their e and dR (one scale a chunk cost less, 124 against 131 us for the gradients of 16 heads x
// 4096 tokens at K = V = 64, 214 against 216 us at 128, and lost the rows 2^-40 below the largest).
template <class KP, int NW>
__device__ __forceinline__ void keep_rows(const f32x4 (&E)[4], const float (&most)[NW][64], uint8_t *base, float *inv,
                                          int col, int grp, int r)
{
    const int tok = scale_token(grp, r);
    uint32_t x = __float_as_uint(most[0][tok]);
#pragma unroll
    for (int w = 1; w < NW; ++w) x = max(x, __float_as_uint(most[w][tok]));
    const Scale f = scale_for(__uint_as_float(x));
    const auto rs = kda::buffer_rsrc(base, KP::BYTES);
    auto put = [&](auto tile) {
        constexpr int t = decltype(tile)::value;
        const f32x4 s = {kda::row_bcast<4 * t>(f.f), kda::row_bcast<4 * t + 1>(f.f), kda::row_bcast<4 * t + 2>(f.f),
                         kda::row_bcast<4 * t + 3>(f.f)};
        kda::bstore8<0>(rs, KP::row_at(col, 16 * t + 4 * grp), 0,
                        __builtin_bit_cast(uint2, kda::to_f16x4(E[t] * s)));
    };
    put(std::integral_constant<int, 0>());
    put(std::integral_constant<int, 1>());
    put(std::integral_constant<int, 2>());
    put(std::integral_constant<int, 3>());
    if (threadIdx.x < 64) inv[tok] = f.inv;
}

// One segment: its sequence, its place in it, and its chunks [c0, c1).
struct Segment {
    int s, i, count, c0, c1;
    __device__ __forceinline__ bool last() const { return i == count - 1; }
};

// Slot -> segment; false where the slot holds none (a sequence without tokens has one, empty segment, so
// that its state is passed on). Binary search as in locate_slot.
__device__ __forceinline__ bool locate_segment(const SeqGeom &sg, int chunks, int slot, Segment *out) {
    const int64_t len = (int64_t)CT * chunks;
    int lo = 0, hi = sg.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (kda::seq_bos(sg, mid) / len + mid <= slot) lo = mid; else hi = mid - 1;
    }
    const int64_t bos = kda::seq_bos(sg, lo), n = (kda::seq_eos(sg, lo, bos) - bos + CT - 1) / CT;
    const int64_t i = slot - (bos / len + lo), count = n > 0 ? (n + chunks - 1) / chunks : 1;
    if (i < 0 || i >= count) return false;
    const int64_t c1 = (i + 1) * chunks;
    *out = Segment{lo, (int)i, (int)count, (int)(i * chunks), (int)(c1 < n ? c1 : n)};
    return true;
}

// The whole sequence as one segment.
__device__ __forceinline__ Segment whole_sequence(const SeqGeom &sg, int s) {
    const int64_t bos = kda::seq_bos(sg, s);
    return Segment{s, 0, 1, 0, (int)((kda::seq_eos(sg, s, bos) - bos + CT - 1) / CT)};
}

// The chunks [c0, c1) of one (sequence, value head) for the C columns from `cbase` of `ld` columns,
// one wave per 16 columns of C.
// init: the state's first element at c0 (row-major, `ld` columns), null for zeros (PHI: ignored);
// end: where to put the end state, or null.
template <int K, int V, int C, int IN, int X, class R, Mode M>
__device__ __forceinline__ void forward_chain(const Params &p, int s, int j, int c0, int c1, int cbase,
                                              const float *init, float *end, uint8_t *lds,
                                              uint8_t *keep = nullptr, Maxima<C / 16> *mx = nullptr)
{
    using L = Stage<K, C, IN, R, M>;
    static_assert(L::BYTES * L::BUFS <= 160 * 1024, "LDS of a compute unit");
    constexpr int NW = C / 16, NT = K / 16, LD = M == PHI ? K : V, NS = K / 32;
    const int tid = threadIdx.x, lane = tid & 63, grp = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = j / p.G;
    const int64_t bos = kda::seq_bos(p.seq, s), eos = kda::seq_eos(p.seq, s, bos);
    const size_t slot0 = (size_t)j * p.seq.n_slots + bos / CT + s;
    const int col0 = 16 * wave;             // within the workgroup's columns

    const RowStage<K, NW> qk_rows((int64_t)p.H * K, wave, lane);
    const RowStage<C, NW> v_rows((int64_t)p.HV * V, wave, lane);
    auto stage = [&](int c, uint8_t *buf) {
        const int64_t t0 = bos + (int64_t)CT * c;
        const int nv = (int)(eos - t0 < CT ? eos - t0 : CT);
        const int64_t qk = (t0 * p.H + h) * K;
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            qk_rows(p.k[i] + qk, nv, buf + L::KM + i * L::MK, wave);
            if constexpr (M == OUT) qk_rows(p.q[i] + qk, nv, buf + L::QM + i * L::MK, wave);
        }
        if constexpr (IN == 1 && M != PHI)
            v_rows((const uint16_t *)p.v + (t0 * p.HV + j) * V + cbase, nv, buf + L::VM, wave);
        stage_block<L::KIB, NW>(p.rec + (slot0 + c) * R::BYTES, buf + L::REC, wave, lane);
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
    for (int t = 0; t < 4; ++t)
        E[t] = zero4();
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
        uint8_t *const buf = lds + ((c - c0) % L::BUFS) * L::BYTES;
        const int64_t t0 = bos + (int64_t)CT * c;
        const int nv = (int)(eos - t0 < CT ? eos - t0 : CT);
        if constexpr (M == KEEP) {
            const float a = largest(S);
            if (lane == 0) mx->state[c & 1][wave] = a;
            mx->rows[c & 1][wave][scale_token(grp, r)] = largest_of_tokens(E, r);
        }
        kda::vm_drain();                    // chunk c has arrived (all of this wave's copies)
        __syncthreads();
        if (L::BUFS == 2 && c + 1 < c1) stage(c + 1, lds + ((c + 1 - c0) % L::BUFS) * L::BYTES);
        if constexpr (M == KEEP) {          // S of this chunk, e of the one before
            float *const inv = (float *)(kept(c) + KP::SCALE);
            keep_state<KP>(S, mx->scale(mx->state[c & 1]), kept(c) + KP::S, inv, cbase + col0 + r, grp);
            if (c > c0)
                keep_rows<KP>(E, mx->rows[c & 1], kept(c - 1) + KP::E, (float *)(kept(c - 1) + KP::SCALE) + KP::SE,
                              cbase + col0 + r, grp, r);
        }
        const uint8_t *const rec = buf + L::REC;
        const float *const ra = (const float *)(rec + R::RA), *const rb = (const float *)(rec + R::RB);
        const float eg = *(const float *)(rec + R::EG);
        // Operands are read from LDS a phase ahead of the products that take them (AHEAD; the reads of
        // a phase fit the registers for one plane only): the compiler by itself reads each operand
        // right before its product and waits.
        constexpr bool AHEAD = IN == 1;
        auto phase = [] { __builtin_amdgcn_sched_barrier(0); };
        Parts<IN> kf[AHEAD ? NS : 1][4], qf[AHEAD && M == OUT ? NS : 1][4];
        auto read_kq = [&](int st, Parts<IN> (&kk)[4], Parts<IN> (&qq)[4]) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int at = piece_at<K>(16 * t + r, 4 * st + grp);
                kk[t] = lds_parts<IN>(buf + L::KM + at, L::MK);
                if constexpr (M == OUT) qq[t] = lds_parts<IN>(buf + L::QM + at, L::MK);
            }
        };
        Parts<X> af[6];
        f32x4 a4[4], v4[4];
        auto read_av = [&] {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                a4[t] = *(const f32x4 *)(ra + 16 * t + 4 * grp);
                v4[t] = zero4();
                if constexpr (M == PHI) {
                } else if constexpr (IN == 1) {
                    v4[t] = widen(lds_tr(buf + L::VM + piece_at<C>(16 * t + 4 * grp + (r >> 2), col0 / 8 + ((r & 3) >> 1)) +
                                         8 * (r & 1)));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = 16 * t + 4 * grp + i;
                        v4[t][i] = ((const float *)p.v)[((t0 + (row < nv ? row : nv - 1)) * p.HV + j) * V + cbase + col0 + r];
                    }
                }
            }
#pragma unroll
            for (int f = 0; f < 6; ++f) af[f] = lds_parts<X>(rec + R::A + f * R::FR + lane * 16, R::MAT);
        };
        Parts<IN> ktf[AHEAD ? 2 : 1][AHEAD ? NT : 1];
        f32x4 b4[4];
        auto read_kt = [&](int st, int t) {
            const int row = 32 * st + 4 * grp + (r >> 2), piece = 4 * (t / 2) + (r & 3), half = 8 * (t % 2);
            const int at0 = piece_at<K>(row, piece) + half, at1 = piece_at<K>(row + 16, piece) + half;
            Parts<IN> kt;
#pragma unroll
            for (int i = 0; i < IN; ++i)
                kt.p[i] = join(lds_tr(buf + L::KM + i * L::MK + at0), lds_tr(buf + L::KM + i * L::MK + at1));
            return kt;
        };
        auto read_kts = [&](int st) {
            if constexpr (AHEAD) {
#pragma unroll
                for (int t = 0; t < NT; ++t) ktf[st][t] = read_kt(st, t);
            }
            b4[2 * st] = *(const f32x4 *)(rb + 32 * st + 4 * grp);
            b4[2 * st + 1] = *(const f32x4 *)(rb + 32 * st + 16 + 4 * grp);
        };

        f32x4 kS[4], O[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            kS[t] = O[t] = zero4();
        if constexpr (AHEAD) {
#pragma unroll
            for (int st = 0; st < NS; ++st) read_kq(st, kf[st], qf[M == OUT ? st : 0]);
            phase();
        }
        // K S and (Q S)^T
#pragma unroll
        for (int st = 0; st < NS; ++st) {
            if constexpr (!AHEAD) read_kq(st, kf[0], qf[0]);
            if (AHEAD && st == NS - 1) {
                phase();
                read_av();
                phase();
            }
            const Parts<X> sp = split<X>(S[2 * st], S[2 * st + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                kS[t] = mm(kf[AHEAD ? st : 0][t], sp, kS[t]);
                if constexpr (M == OUT) O[t] = mm(sp, qf[AHEAD ? st : 0][t], O[t]);
            }
        }
        if constexpr (!AHEAD) read_av();
        phase();
        read_kts(0);
        phase();
#pragma unroll
        for (int t = 0; t < NT; ++t)
            S[t] *= eg;
        // R = V - e^Gam (K S), as operands; e = A R
        Parts<X> rp[2];
#pragma unroll
        for (int st = 0; st < 2; ++st)
            rp[st] = split<X>(v4[2 * st] - a4[2 * st] * kS[2 * st],
                              v4[2 * st + 1] - a4[2 * st + 1] * kS[2 * st + 1]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            E[t] = mm(af[frag_index(t, 0)], rp[0], zero4());
            if (t >= 2) E[t] = mm(af[frag_index(t, 1)], rp[1], E[t]);
        }
        phase();
        read_kts(1);
        phase();
        Parts<X> mf[6];
        if constexpr (M == OUT && AHEAD) {
#pragma unroll
            for (int f = 0; f < 6; ++f) mf[f] = lds_parts<X>(rec + R::M + f * R::FR + lane * 16, R::MAT);
            phase();
        }
        // S += K^T (beta e^{gam - Gam} e)
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const Parts<X> dp = split<X>(b4[2 * st] * E[2 * st], b4[2 * st + 1] * E[2 * st + 1]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const Parts<IN> kt = AHEAD ? ktf[AHEAD ? st : 0][AHEAD ? t : 0] : read_kt(st, t);
                S[t] = mm(kt, dp, S[t]);
            }
        }
        if constexpr (M == OUT) {           // o = scale e^Gam (Q S) + M e
            const float *const rc = (const float *)(rec + R::RC);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                O[t] *= rc[16 * t + r];
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                const Parts<X> ep = split<X>(E[2 * st], E[2 * st + 1]);
#pragma unroll
                for (int t = 2 * st; t < 4; ++t) {
                    const int f = frag_index(t, st);
                    const Parts<X> m = AHEAD ? mf[f] : lds_parts<X>(rec + R::M + f * R::FR + lane * 16, R::MAT);
                    O[t] = mm(ep, m, O[t]);
                }
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
            mx->rows[c1 & 1][wave][scale_token(grp, r)] = largest_of_tokens(E, r);
            __syncthreads();
            keep_rows<KP>(E, mx->rows[c1 & 1], kept(c1 - 1) + KP::E, (float *)(kept(c1 - 1) + KP::SCALE) + KP::SE,
                          cbase + col0 + r, grp, r);
        }
    }
    if (end) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                end[(size_t)state_row(t, i, grp) * LD + cbase + col0 + r] = S[t][i];
        if constexpr (M == PHI) {           // and the transpose behind it
            const auto rs = kda::buffer_rsrc(end + K * K, K * K * 4);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                kda::bstore16<0>(rs, ((cbase + col0 + r) * K + state_row(t, 0, grp)) * 4, 0, S[t]);
        }
    }
}

}  // namespace gdn
