// gdn_backward.hip -- gradients of the gated delta rule, bf16 io (gdn_internal.h has the forward's
// chunk formulas; matrices and row scales as there, dS' the gradient of the state at a chunk's end).
//
// Per chunk, newest first, the state's gradient goes through
//     de = M^T dO + beta e^{gam-Gam} . (K dS')        dR = A^T de   (= dV)
//     dS = e^gam dS' + Q^T (scale e^Gam . dO) - K^T (e^Gam . dR)
// and every chunk then gives its tokens, from S at its start, dS', e and dR alone,
//     X1 = lower(dO e^T),  X2 = -strictly_lower(dR e^T)      (gradients of M and L)
//     dQ = (X1 . scale D beta_j) K + scale e^Gam . (dO S^T)
//     dK = (X1 . scale D beta_j)^T Q + (W2 + W2^T) K - e^Gam . (dR S^T) + beta T,  W2 = X2 . D beta_j,
//     T_j = e^{gam-Gam_j} dS' e_j
//     dbeta_j = sum_i U_ij + k_j.T_j,   U = D . (X1 . scale Q K^T + X2 . K K^T)
//     dg_t = sum_{i >= t > j} beta_j U_ij + sum_{i >= t} (q_i.dQ_i[S part] + k_i.dK_i[S part])
//            + sum_{j < t} beta_j k_j.T_j + e^gam <S, dS'>.
// (dg_t is what crosses t: every term holds a decay over t. As differences of row and column sums
// the pairs on one side of t would cancel only to rounding, which a strong decay at t would show.)
// No division by beta and no exponent above zero occurs.
//
// Launches: the chunk records (gdn_prepare.hip), both passes over the chunks (the forward one for
// S and e, the reverse one for dS' and dR; they are independent, one launch), the chunks' tokens.
// The passes carry two bf16 parts of every operand as the forward does (dh0 is an fp32 result).
// What they leave for the chunks is scaled fp16 (2^-11 a rounding, against the 2^-8 of the bf16
// gradients that it enters; bf16 there cost up to 5e-3 of dg, whose terms cancel), multiplied with
// dO as fp16 (bf16 values scaled by a power of two a token: exact down to 2^-28 of the token's largest); the
// 64 x 64 matrices take two bf16 parts against the stored q and k.
//
// Measured, 16 heads x 4096 tokens, K = V = 128: records 17 us, segments' ends 57, their joining 15, both
// passes 57, tokens 72 (216 for the call repeated, 229 with inputs that change; without segments and with four
// 64 x 64 matrices 519). The passes are bound by a chunk's dependent products with two waves a SIMD (7 us a chunk
// with every compute unit busy: vector instructions issue 41% of it, LDS works 30%, the matrix core 25%). The
// tokens' kernel has one workgroup a compute unit, which takes 37 thousand clocks; vector instructions issue in 20
// of them, LDS works 12 (4 of bank conflicts) and the matrix core 4: the phases between its barriers wait for each
// other. By timestamps 8 thousand go to loading, 6 to forming the matrices, 9 to the products with the states.
#include <type_traits>

#include "gdn_segments.h"

namespace gdn {

namespace {

template <int K, int C>
struct StageR {                             // LDS of one chunk of the reverse pass
    static constexpr int MK = 64 * K * 2, MV = 64 * C * 2;
    static constexpr int KM = 0, QM = MK, DO = 2 * MK, REC = DO + MV;
    static constexpr int BYTES = REC + RecB::REV_KIB * 1024;
};

// The reverse pass over chunks c1 - 1 .. c0 for the C columns from `cbase`, from the gradient `init` of the
// state behind them (null: zero) to the gradient `end` of the state before them (or null). KEPT: leaves dS'
// and dR for the local kernel (all columns in one workgroup then, for the scales); else a segment's end only.
template <int K, int V, int C, int BUFS, bool KEPT>
__device__ __forceinline__ void reverse_chain(const BwdParams &b, int s, int j, int c0, int c1, int cbase,
                                              const float *init, float *end, uint8_t *lds,
                                              Maxima<C / 16> *mx = nullptr)
{
    using L = StageR<K, C>;
    using R = RecB;
    using KP = Keep<K, V>;
    constexpr int X = R::X, NW = C / 16, NT = K / 16;
    const Params &p = b.f;
    const int tid = threadIdx.x, lane = tid & 63, grp = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = j / p.G;
    const int64_t bos = kda::seq_bos(p.seq, s), eos = kda::seq_eos(p.seq, s, bos);
    const size_t slot0 = (size_t)j * p.seq.n_slots + bos / CT + s;
    const int col0 = 16 * wave;

    const RowStage<K, NW> qk_rows((int64_t)p.H * K, wave, lane);
    const RowStage<C, NW> v_rows((int64_t)p.HV * V, wave, lane);
    auto stage = [&](int c, uint8_t *buf) {
        const int64_t t0 = bos + (int64_t)CT * c;
        const int nv = (int)(eos - t0 < CT ? eos - t0 : CT);
        const int64_t qk = (t0 * p.H + h) * K;
        qk_rows(p.k[0] + qk, nv, buf + L::KM, wave);
        qk_rows(p.q[0] + qk, nv, buf + L::QM, wave);
        v_rows(b.d_o + (t0 * p.HV + j) * V + cbase, nv, buf + L::DO, wave);
        stage_block<R::REV_KIB, NW>(p.rec + (slot0 + c) * R::BYTES + R::REV, buf + L::REC, wave, lane);
    };
    if (c0 < c1) stage(c1 - 1, lds);
    auto kept = [&](int c) { return b.keep + (slot0 + c) * KP::BYTES; };

    f32x4 S[NT], D[4];                      // dS, laid out as the forward's S; dR
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[t][i] = init ? init[(size_t)state_row(t, i, grp) * V + cbase + col0 + r] : 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t) D[t] = zero4();

#pragma unroll 1
    for (int c = c1 - 1; c >= c0; --c) {
        uint8_t *const buf = lds + (c1 - 1 - c) % BUFS * L::BYTES;
        if constexpr (KEPT) {
            const float x = largest(S);
            if (lane == 0) mx->state[c & 1][wave] = x;
            mx->rows[c & 1][wave][scale_token(grp, r)] = largest_of_tokens(D, r);
        }
        kda::vm_drain();
        __syncthreads();
        if (BUFS == 2 && c > c0) stage(c - 1, lds + (c1 - c) % BUFS * L::BYTES);
        if constexpr (KEPT) {
        keep_state<KP>(S, mx->scale(mx->state[c & 1]), kept(c) + KP::DS, (float *)(kept(c) + KP::SCALE) + 1, col0 + r, grp);
        if (c < c1 - 1)
            keep_rows<KP>(D, mx->rows[c & 1], kept(c + 1) + KP::DR, (float *)(kept(c + 1) + KP::SCALE) + KP::SR,
                          col0 + r, grp, r);
        }
        const uint8_t *const rec = buf + L::REC - R::REV;
        const float *const ra = (const float *)(rec + R::RA), *const rb = (const float *)(rec + R::RB),
                    *const rc = (const float *)(rec + R::RC);
        const float eg = *(const float *)(rec + R::EG);
        // K dS'
        f32x4 kS[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) kS[t] = zero4();
#pragma unroll
        for (int st = 0; st < K / 32; ++st) {
            const Parts<X> sp = split<X>(S[2 * st], S[2 * st + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                kS[t] = mm(Parts<1>{lds_b128(buf + L::KM + piece_at<K>(16 * t + r, 4 * st + grp))}, sp, kS[t]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) S[t] *= eg;
        // de = M^T dO + beta e^{gam-Gam} (K dS'); dO of tokens 32 st + 4 g .. + 3, + 16 per lane
        s16x4 dv[2][2];
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                dv[st][u] = lds_tr(buf + L::DO + piece_at<C>(32 * st + 16 * u + 4 * grp + (r >> 2),
                                                             col0 / 8 + ((r & 3) >> 1)) + 8 * (r & 1));
        Parts<X> dp[2];
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            f32x4 x[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = 2 * st + u;
                x[u] = *(const f32x4 *)(rb + 16 * t + 4 * grp) * kS[t];
#pragma unroll
                for (int s2 = st; s2 < 2; ++s2)
                    x[u] = mm(lds_parts<X>(rec + R::MT + frag_index_t(t, s2) * R::FR + lane * 16, R::MAT),
                              Parts<1>{join(dv[s2][0], dv[s2][1])}, x[u]);
            }
            dp[st] = split<X>(x[0], x[1]);
        }
        // dR = A^T de
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            D[t] = zero4();
#pragma unroll
            for (int st = t / 2; st < 2; ++st)
                D[t] = mm(lds_parts<X>(rec + R::AT + frag_index_t(t, st) * R::FR + lane * 16, R::MAT), dp[st], D[t]);
        }
        // dS = e^gam dS' + Q^T (scale e^Gam dO) - K^T (e^Gam dR)
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const f32x4 a0 = *(const f32x4 *)(ra + 32 * st + 4 * grp), a1 = *(const f32x4 *)(ra + 32 * st + 16 + 4 * grp);
            const f32x4 c0v = *(const f32x4 *)(rc + 32 * st + 4 * grp), c1v = *(const f32x4 *)(rc + 32 * st + 16 + 4 * grp);
            const Parts<X> rp = split<X>(zero4() - a0 * D[2 * st], zero4() - a1 * D[2 * st + 1]),
                           op = split<X>(c0v * widen(dv[st][0]), c1v * widen(dv[st][1]));
            const int row = 32 * st + 4 * grp + (r >> 2);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int piece = 4 * (t / 2) + (r & 3), half = 8 * (t % 2);
                const int at0 = piece_at<K>(row, piece) + half, at1 = piece_at<K>(row + 16, piece) + half;
                S[t] = mm(Parts<1>{join(lds_tr(buf + L::KM + at0), lds_tr(buf + L::KM + at1))}, rp, S[t]);
                S[t] = mm(Parts<1>{join(lds_tr(buf + L::QM + at0), lds_tr(buf + L::QM + at1))}, op, S[t]);
            }
        }
        if (BUFS == 1 && c > c0) {
            __syncthreads();                // every wave is done with the buffer
            stage(c - 1, lds);
        }
    }
    if (KEPT && c0 < c1) {
        mx->rows[(c0 - 1) & 1][wave][scale_token(grp, r)] = largest_of_tokens(D, r);
        __syncthreads();
        keep_rows<KP>(D, mx->rows[(c0 - 1) & 1], kept(c0) + KP::DR, (float *)(kept(c0) + KP::SCALE) + KP::SR,
                      col0 + r, grp, r);
    }
    if (end) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) end[(size_t)state_row(t, i, grp) * V + cbase + col0 + r] = S[t][i];
    }
}

}  // namespace

// Both passes: parts 0 and 1 of a unit (SEG: of a segment).
template <int K, int V, bool SEG>
__global__ __launch_bounds__(V * 4) void chains_kernel(BwdParams b)
{
    using F = Stage<K, V, 1, RecB, KEEP>;
    constexpr int FB = F::BYTES * F::BUFS, RB = 2 * StageR<K, V>::BYTES, BYTES = FB > RB ? FB : RB;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[BYTES];
    __shared__ Maxima<V / 16> mx;
    static_assert(BYTES + sizeof(mx) <= 160 * 1024, "LDS of a compute unit");
    const Params &p = b.f;
    constexpr size_t KV = (size_t)K * V;
    int unit, part;
    if (!unit_of(blockIdx.x, 2, (SEG ? p.seg.slots : p.seq.N) * p.HV, &unit, &part)) return;
    Segment g;
    if constexpr (SEG) {
        if (!locate_segment(p.seq, p.seg.chunks, unit / p.HV, &g)) return;
    } else {
        unit = kda::longest_first(p.seq, p.HV, unit);
        g = whole_sequence(p.seq, unit / p.HV);
    }
    const int j = unit % p.HV;
    const size_t at = ((size_t)g.s * p.HV + j) * KV;
    if (part == 0) {
        const float *const init = SEG ? segment_start<K, V>(p, g, unit / p.HV, j) : p.h0 ? p.h0 + at : nullptr;
        forward_chain<K, V, V, 1, RecB::X, RecB, KEEP>(p, g.s, j, g.c0, g.c1, 0, init, nullptr, lds, b.keep, &mx);
    } else {
        const float *const init = !g.last() ? p.seg.G + ((size_t)unit + p.HV) * KV : b.dht ? b.dht + at : nullptr;
        reverse_chain<K, V, V, 2, true>(b, g.s, j, g.c0, g.c1, 0, init, g.i == 0 && b.dh0 ? b.dh0 + at : nullptr, lds, &mx);
    }
}

// The first pass over segments: E and PHI (gdn_segments.h), and G of every segment but the first.
template <int K, int V>
__global__ __launch_bounds__(256, 2) void bwd_ends_kernel(BwdParams b)
{
    using LE = Stage<K, 64, 1, RecB, END>;
    using LP = Stage<K, 64, 1, RecB, PHI>;
    constexpr int A = LE::BYTES * LE::BUFS, B = LP::BYTES * LP::BUFS, G = StageR<K, 64>::BYTES;
    constexpr int AB = A > B ? A : B, NF = V / 64 + K / 64, NP = NF + V / 64;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[AB > G ? AB : G];
    const Params &p = b.f;
    int unit, part;
    if (!unit_of(blockIdx.x, NP, p.seg.slots * p.HV, &unit, &part)) return;
    const int j = unit % p.HV;
    if (part < NF) {
        forward_ends<K, V, 1, RecB::X, RecB>(p, unit / p.HV, j, part, lds);
        return;
    }
    Segment g;
    if (!locate_segment(p.seq, p.seg.chunks, unit / p.HV, &g) || g.i == 0) return;
    const float *const init = g.last() && b.dht ? b.dht + ((size_t)g.s * p.HV + j) * K * V : nullptr;
    reverse_chain<K, V, 64, 1, false>(b, g.s, j, g.c0, g.c1, 64 * (part - NF), init, p.seg.G + (size_t)unit * K * V, lds);
}

template <int K, int V>
__global__ __launch_bounds__(256) void bwd_join_kernel(Params p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[Join<K, RecB::X>::BYTES];
    int unit, part;
    if (!unit_of(blockIdx.x, V / 8, p.seq.N * p.HV, &unit, &part)) return;
    const int s = unit / p.HV, j = unit % p.HV;
    if (part & 1)
        join_ends<K, V, RecB::X, true>(p, p.seg.G, s, j, part / 2 * 16, lds);
    else
        join_ends<K, V, RecB::X, false>(p, p.seg.E, s, j, part / 2 * 16, lds);
}

namespace {

// LDS of the local kernel. The two 64 x 64 matrices (128-byte rows, pieces swizzled) lie where the state
// was, once its products are done.
template <int K, int V>
struct Local {
    static constexpr int MK = 64 * K * 2, MV = 64 * V * 2, MS = V * K * 2;
    static constexpr int Q = 0, KM = MK, DO = 2 * MK, E = DO + MV, DR = E + MV, S = DR + MV, DS = S + MS;
    static constexpr int W = S;             // P1, P2 [j][i], two parts each
    static constexpr int SCAL = DS + MS > W + 4 * 8192 ? DS + MS : W + 4 * 8192;
    static constexpr int INV = SCAL + 2048, END = INV + 1024;   // RecB's scalars, Keep's scales
};

template <int ND, int NW>
struct LocalScalars {
    float rowsum[4][64], colsum[4][64];     // of beta_j U, U below the diagonal, per tile column / row
    float diag[64];                         // of U
    float cross[64];                        // sum_{i >= t > j} beta_j U_ij within t's own tile
    float qs[ND][64], ks[ND][64], kt[ND][64];   // per 16 key dims: q.dQ[S part], k.dK[S part], k.T
    float sd[NW];                           // per wave: <S, dS'>
    float so[64];                           // what undoes the scale of a token's dO
    float dot[2][ND][64];                   // per 16 key dims: q.dq, k.dk (L2 norm)
};

// The largest of 8 or 16 neighbouring lanes' values (every one gets it).
template <int N>
__device__ __forceinline__ uint32_t row_max(uint32_t u) {
    u = max(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0xb1, 0xf, 0xf, false));    // quad_perm 1,0,3,2
    u = max(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x4e, 0xf, 0xf, false));    // quad_perm 2,3,0,1
    u = max(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x141, 0xf, 0xf, false));   // row_half_mirror
    if (N == 16) u = max(u, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x140, 0xf, 0xf, false));  // row_mirror
    return u;
}

// Within 16 lanes: the sum of the lanes before this one, and of this one and those behind it.
__device__ __forceinline__ float row_shift(float x) {      // the value of the lane before, or zero
    return __builtin_amdgcn_update_dpp(0.f, x, 0x111, 0xf, 0xf, false);
}
__device__ __forceinline__ float row_before(float x) { return row_shift(kda::row_inclusive_scan(x)); }
__device__ __forceinline__ float lane_of(float x, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}
__device__ __forceinline__ float row_from(float x) {
    x += __builtin_amdgcn_update_dpp(0.f, x, 0x101, 0xf, 0xf, false);   // row_shl:1
    x += __builtin_amdgcn_update_dpp(0.f, x, 0x102, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0.f, x, 0x104, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0.f, x, 0x108, 0xf, 0xf, false);
    return x;
}

__device__ __forceinline__ int w_at(int row, int piece) { return piece_at<64>(row, piece); }

}  // namespace

// One workgroup per (chunk slot, q/k head), over the head's value heads, one wave per 16 key dims and half
// of the tokens: dQ and dK stay in registers, transposed (a lane: four consecutive dims of one token). A
// chunk fills the LDS of a compute unit, so the waves of one workgroup are all there is to hide latencies:
// 16 waves took 78 us for 16 heads x 4096 tokens, eight waves with all tokens each 81 us (first calls).
template <int K, int V>
__global__ __launch_bounds__(K * 8) void local_kernel(BwdParams b)
{
    using L = Local<K, V>;
    using R = RecB;
    constexpr int ND = K / 16, NW = 2 * ND, NTH = 64 * NW, NL = 8;  // NL: waves that copy to LDS
    __shared__ __attribute__((aligned(1024))) uint8_t lds[L::END];
    __shared__ __attribute__((aligned(16))) LocalScalars<ND, NW> sc;
    static_assert(L::END + sizeof(sc) <= 160 * 1024, "LDS of a compute unit");
    const Params &p = b.f;
    const int tid = threadIdx.x, lane = tid & 63;
    int grp = lane >> 4, r = lane & 15;
    // LDS addresses are cheap to form and many: without this the compiler forms those of every
    // phase ahead of the loop over the heads and keeps them in (spilled) registers
    auto new_phase = [&] {
        asm volatile("" : "+v"(grp), "+v"(r));
        __builtin_amdgcn_sched_barrier(0);
    };
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int dims = wave % ND, half = wave / ND;   // this wave's key dims 16 dims .., token tiles 2 half ..
    const int slot = blockIdx.x, h = blockIdx.y;
    int s, nv;
    int64_t bos;
    if (!kda::locate_slot<CT>(p.seq, slot, &s, &bos, &nv)) return;
    const float *const scal = (const float *)(lds + L::SCAL);
    const float *const ghi = scal, *const glo = scal + 64, *const beta = scal + 128, *const rk = scal + 192,
                *const rq = scal + 256;
    const int64_t qk0 = (bos * p.H + h) * K;
    if (wave < NL) {
        stage_rows<K, NL>(p.q[0] + qk0, (int64_t)p.H * K, nv, lds + L::Q, wave, lane);
        stage_rows<K, NL>(p.k[0] + qk0, (int64_t)p.H * K, nv, lds + L::KM, wave, lane);
    }

    using KP = Keep<K, V>;
    // operand of this wave's 16 key dims, k = 32 columns from `c0` of a kept state
    auto state_a = [&](int base, int c0) {
        const int col = c0 + 8 * grp + (r >> 2), dim = 16 * dims + 4 * (r & 3);
        return join(lds_tr(lds + base + KP::state_at(col, dim)), lds_tr(lds + base + KP::state_at(col + 4, dim)));
    };
    // and k = 32 rows from `row0` of q or k
    auto dims_a = [&](int base, int row0) {
        const int row = row0 + 8 * grp + (r >> 2), piece = 2 * dims + ((r & 3) >> 1);
        return join(lds_tr(lds + base + piece_at<K>(row, piece) + 8 * (r & 1)),
                    lds_tr(lds + base + piece_at<K>(row + 4, piece) + 8 * (r & 1)));
    };
    auto half8 = [](bf16x8 x) { return __builtin_bit_cast(kda::f16x8, x); };
    // operand of 16 tokens from `tok0`, k = 32 columns from `c0` of e or dR
    auto toks_t = [&](int base, int c0, int tok0) {
        const int col = c0 + 8 * grp + (r >> 2), tok = tok0 + 4 * (r & 3);
        return join(lds_tr(lds + base + KP::row_at(col, tok)), lds_tr(lds + base + KP::row_at(col + 4, tok)));
    };
    auto row_of = [&](int base, int t) {            // four dims of token 16 t + r of q or k
        const int d = 16 * dims + 4 * grp;
        f32x4 x;
        kda::unpack_bf16x4(*(const uint2 *)(lds + base + piece_at<K>(16 * t + r, d / 8) + 2 * (d & 4)), (float *)&x);
        return x;
    };
    auto dot4 = [](f32x4 a, f32x4 c) { return a[0] * c[0] + a[1] * c[1] + a[2] * c[2] + a[3] * c[3]; };

    f32x4 dq[2], dk[2];                             // [token tile]
#pragma unroll
    for (int u = 0; u < 2; ++u) dq[u] = dk[u] = zero4();

#pragma unroll 1
    for (int m = 0; m < p.G; ++m) {
        const int j = h * p.G + m;
        const size_t at = (size_t)j * p.seq.n_slots + slot;
        const uint8_t *const keep = b.keep + at * KP::BYTES;
        if (m > 0) __syncthreads();                 // the previous head is done with the buffers
        static_assert(L::DR == L::E + L::MV && L::DS == L::S + L::MS, "copied as they are stored");
        constexpr int LATE = 2 * L::MS / 1024 / NL;     // copies of the states, a wave
        if (wave < NL) {
            stage_block<2, NL>(p.rec + at * R::BYTES + R::GHI, lds + L::SCAL, wave, lane);
            stage_rows<V, NL>(b.d_o + (bos * p.HV + j) * V, (int64_t)p.HV * V, nv, lds + L::DO, wave, lane);
            // e, dR and the scales; the states last, as they are used last
            stage_block<2 * L::MV / 1024, NL>(keep + KP::E, lds + L::E, wave, lane);
            if (wave == NL - 1) copy16_to_lds(keep + KP::SCALE, lane * 16, lds + L::INV);
            stage_block<2 * L::MS / 1024, NL>(keep + KP::S, lds + L::S, wave, lane);
        }
        asm volatile("s_waitcnt vmcnt(%0)" :: "n"(LATE) : "memory");
        __syncthreads();
        const float *const inv = (const float *)(lds + L::INV);
        const float fs = inv[0], fds = inv[1];
        const float *const fe = inv + KP::SE, *const fdr = inv + KP::SR, *const so = sc.so;
        const float whi = ghi[63], wlo = glo[63];
        // dO as fp16, in place: a thread a 16-byte piece, the V / 8 threads of a token side by side
#pragma unroll
        for (int q = 0; q < (64 * V / 8 + NTH - 1) / NTH; ++q) {
            const int n = q * NTH + tid;
            if (n >= 64 * V / 8) break;             // (whole waves)
            uint8_t *const piece = lds + L::DO + n * 16;
            const uint4 ob = *(const uint4 *)piece;
            f32x4 x, y;
            kda::unpack_bf16x4(make_uint2(ob.x, ob.y), (float *)&x);
            kda::unpack_bf16x4(make_uint2(ob.z, ob.w), (float *)&y);
            const Scale f = scale_for(__uint_as_float(row_max<V / 8>(__float_as_uint(max_abs(y, max_abs(x, 0.f))))));
            const uint2 a = half4(x, f.f), c = half4(y, f.f);
            *(uint4 *)piece = make_uint4(a.x, a.y, c.x, c.y);
            if (n % (V / 8) == 0) sc.so[n / (V / 8)] = f.inv;
        }
        __syncthreads();

        new_phase();
        // the 64 x 64 matrices, lower tiles n = wave, wave + NW, .. of (0,0) (1,0) (1,1) ...
        constexpr int NU = (10 + NW - 1) / NW;
        f32x4 w1[NU], w2[NU];
        int tis[NU], tjs[NU];
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int n = wave + NW * u;
            const int ti = n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3, tj = n - ti * (ti + 1) / 2;
            tis[u] = ti;
            tjs[u] = tj;
            if (n >= 10) continue;
            f32x4 x1 = zero4(), x2 = zero4(), qk = zero4(), kk = zero4();
#pragma unroll
            for (int st = 0; st < V / 32; ++st) {
                const kda::f16x8 e = half8(toks_t(L::E, 32 * st, 16 * tj));
                x1 = mfma32(half8(lds_b128(lds + L::DO + piece_at<V>(16 * ti + r, 4 * st + grp))), e, x1);
                x2 = mfma32(half8(toks_t(L::DR, 32 * st, 16 * ti)), e, x2);
            }
#pragma unroll
            for (int st = 0; st < K / 32; ++st) {
                const bf16x8 kj = lds_b128(lds + L::KM + piece_at<K>(16 * tj + r, 4 * st + grp));
                qk = mfma32(lds_b128(lds + L::Q + piece_at<K>(16 * ti + r, 4 * st + grp)), kj, qk);
                kk = mfma32(lds_b128(lds + L::KM + piece_at<K>(16 * ti + r, 4 * st + grp)), kj, kk);
            }
            __builtin_amdgcn_sched_barrier(0);
            const int jj = 16 * tj + r;
            const float bj = beta[jj], rkj = rk[jj], fej = fe[jj], fej1 = fej * p.scale;
            float col = 0.f;
            f32x4 bu;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 16 * ti + 4 * grp + e;
                const float d = i >= jj && i < nv
                                    ? __builtin_amdgcn_exp2f((ghi[i] - ghi[jj]) + (glo[i] - glo[jj]))
                                    : 0.f;
                const float y1 = d != 0.f ? x1[e] * so[i] * d * fej1 : 0.f;
                const float y2 = d != 0.f && i > jj ? x2[e] * fdr[i] * d * -fej : 0.f;
                const float uu = rkj * (y1 * rq[i] * qk[e] + y2 * rk[i] * kk[e]);
                if (i == jj) sc.diag[i] = uu;
                col += i > jj ? uu : 0.f;
                float row = i > jj ? bj * uu : 0.f;
                bu[e] = row;
                row = kda::row_inclusive_scan(row);
                if (r == 15) sc.rowsum[tj][i] = row;
                w1[u][e] = y1 * bj * rkj * rq[i];
                w2[u][e] = y2 * bj * rkj * rk[i];
            }
            col = sum_groups(col);
            if (grp == 0) sc.colsum[ti][jj] = col;
            if (ti == tj) {                         // lane column r stands for t: columns j < t of rows i >= t
                float x = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float before = row_before(bu[e]);
                    x += 4 * grp + e >= r ? before : 0.f;
                }
                x = sum_groups(x);
                if (grp == 0) sc.cross[jj] = x;
            }
            new_phase();
        }
        // products with the states: dQ and dK of the S part, T; dq and dk are times rq and rk
        kda::vm_drain();
        __syncthreads();
        float sd = 0.f;
#pragma unroll
        for (int q = 0; q < V * K / 8 / NTH; ++q) {
            const int o = (q * NTH + tid) * 16;
            const kda::f16x8 x = half8(lds_b128(lds + L::S + o)), y = half8(lds_b128(lds + L::DS + o));
#pragma unroll
            for (int e = 0; e < 8; ++e) sd += (float)x[e] * (float)y[e];
        }
        sd *= fs * fds;
        sd = kda::wave_sum(sd);
        if (lane == 0) sc.sd[wave] = sd;
        new_phase();
        f32x4 xs[2], ys[2], zs[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) xs[u] = ys[u] = zs[u] = zero4();
#pragma unroll
        for (int st = 0; st < V / 32; ++st) {
            const kda::f16x8 sa = half8(state_a(L::S, 32 * st)), da = half8(state_a(L::DS, 32 * st));
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = 2 * half + u;
                xs[u] = mfma32(sa, half8(lds_b128(lds + L::DO + piece_at<V>(16 * t + r, 4 * st + grp))), xs[u]);
                ys[u] = mfma32(sa, half8(toks_t(L::DR, 32 * st, 16 * t)), ys[u]);
                zs[u] = mfma32(da, half8(toks_t(L::E, 32 * st, 16 * t)), zs[u]);
            }
        }
        new_phase();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int t = 2 * half + u, i = 16 * t + r;
            const bool live = i < nv;
            const float head = __builtin_amdgcn_exp2f(ghi[i] + glo[i]);
            const float tail = __builtin_amdgcn_exp2f((whi - ghi[i]) + (wlo - glo[i]));
            const f32x4 x = xs[u] * so[i] * (live ? fs * p.scale * head * rq[i] : 0.f),
                        y = ys[u] * fdr[i] * (live ? -fs * head * rk[i] : 0.f),
                        z = zs[u] * fe[i] * (live ? fds * tail * rk[i] : 0.f);
            const f32x4 qr = row_of(L::Q, t), kr = row_of(L::KM, t);
            const float qs = sum_groups(dot4(qr, x)), ks = sum_groups(dot4(kr, y)), kt = sum_groups(dot4(kr, z));
            if (grp == 0) {
                sc.qs[dims][i] = qs;
                sc.ks[dims][i] = ks;
                sc.kt[dims][i] = kt;
            }
            dq[u] += x;
            dk[u] += y + beta[i] * z;
        }
        // dv: four columns of a token per lane, from dR
#pragma unroll
        for (int q = 0; q < V / 4 / NW; ++q) {      // 4 token tiles x V / 16 column tiles
            const int job = q * NW + wave, t = job & 3, c0 = 16 * (job >> 2);
            const s16x4 x = lds_tr(lds + L::DR + KP::row_at(c0 + 4 * grp + (r >> 2), 16 * t + 4 * (r & 3)));
            const kda::f16x4 y = __builtin_bit_cast(kda::f16x4, x);
            const f32x4 z = f32x4{(float)y[0], (float)y[1], (float)y[2], (float)y[3]} * fdr[16 * t + r];
            if (16 * t + r < nv)
                *(uint2 *)(b.dv + ((bos + 16 * t + r) * p.HV + j) * V + c0 + 4 * grp) =
                    __builtin_bit_cast(uint2, kda::to_bf16x4(z));
        }
        __syncthreads();                            // S and dS' are read: the matrices take their place
        new_phase();
        uint8_t *const W = lds + L::W;
        auto put = [&](int k, int ti, int tj, f32x4 x) {    // [j][i], a lane's four i of one j
            const int d = 16 * ti + 4 * grp;
            const int to = k * 16384 + w_at(16 * tj + r, d / 8) + 2 * (d & 4);
            const kda::bf16x4 hi = kda::to_bf16x4(x);
            kda::bf16x4 lo;
#pragma unroll
            for (int e = 0; e < 4; ++e) lo[e] = (__bf16)(x[e] - (float)hi[e]);
            *(uint2 *)(W + to) = __builtin_bit_cast(uint2, hi);
            *(uint2 *)(W + to + 8192) = __builtin_bit_cast(uint2, lo);
        };
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            if (wave + NW * u >= 10) continue;
            const int ti = tis[u], tj = tjs[u];
            put(0, ti, tj, w1[u]);
            put(1, ti, tj, w2[u]);
        }
        if (wave >= NW - 2) {                       // the tiles above the diagonal that are read
            const int ti = wave == NW - 2 ? 0 : 2;
#pragma unroll
            for (int k = 0; k < 2; ++k) put(k, ti, ti + 1, zero4());
        }
        __syncthreads();
        // [j][i] matrix k as operand: 16 columns i of tile t over 32 rows j, or 16 rows j over 32 i
        auto cols = [&](int k, int t, int st) {
            const int row = 32 * st + 8 * grp + (r >> 2), piece = 2 * t + ((r & 3) >> 1), half = 8 * (r & 1);
            const uint8_t *const a = W + k * 16384 + w_at(row, piece) + half,
                          *const c = W + k * 16384 + w_at(row + 4, piece) + half;
            return Parts<2>{join(lds_tr(a), lds_tr(c)), join(lds_tr(a + 8192), lds_tr(c + 8192))};
        };
        auto rows = [&](int k, int t, int st) {
            return lds_parts<2>(W + k * 16384 + w_at(16 * t + r, 4 * st + grp), 8192);
        };
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const Parts<1> qa = {dims_a(L::Q, 32 * st)}, ka = {dims_a(L::KM, 32 * st)};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = 2 * half + u;
                if (st <= half) {
                    dq[u] = mm(ka, cols(0, t, st), dq[u]);
                    dk[u] = mm(ka, cols(1, t, st), dk[u]);
                }
                if (st >= half) {
                    dk[u] = mm(qa, rows(0, t, st), dk[u]);
                    dk[u] = mm(ka, rows(1, t, st), dk[u]);
                }
            }
            new_phase();
        }
        if (wave == 0) {                            // dbeta and dg, a token per lane
            const int i = lane;
            const int tau = i >> 4;
            float left = 0.f, below = 0.f, tiles = 0.f, qsum = 0.f, ksum = 0.f, tsum = 0.f, col = sc.colsum[tau][i];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w < tau) left += sc.rowsum[w][i];       // tiles left of the token's own
                if (w > tau) below += sc.colsum[w][i];      // and below it
            }
            float sd = 0.f;
#pragma unroll
            for (int w = 0; w < ND; ++w) {
                qsum += sc.qs[w][i];
                ksum += sc.ks[w][i];
                tsum += sc.kt[w][i];
            }
#pragma unroll
            for (int w = 0; w < NW; ++w) sd += sc.sd[w];
            // whole tiles that cross: (2,0) and (3,0) for tile 1, (3,0) and (3,1) for tile 2
            const float c0 = row_from(sc.rowsum[0][i]), c1 = row_from(sc.rowsum[1][i < 48 ? 48 : i]);
            const float t20 = lane_of(c0, 32), t30 = lane_of(c0, 48), t31 = lane_of(c1, 48);
            if (tau == 1) tiles = t20 + t30;
            if (tau == 2) tiles = t30 + t31;
            const bool live = i < nv;
            const float bt = beta[i], dbt = col + below + tsum + sc.diag[i];
            const float pairs = sc.cross[i] + row_from(left) + row_before(bt * below) + tiles;
            // the suffix sums of the states' parts and the prefix sums of beta k.T: within 16 lanes, then the
            // other tiles' sums
            const float from = row_from(live ? qsum + ksum : 0.f), upto = kda::row_inclusive_scan(live ? bt * tsum : 0.f);
            float x = pairs + from + row_shift(upto) + __builtin_amdgcn_exp2f(whi + wlo) * sd;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w > tau) x += lane_of(from, 16 * w);
                if (w < tau) x += lane_of(upto, 16 * w + 15);
            }
            if (live) {
                const int64_t o = (bos + i) * p.HV + j;
                const float db = p.pre.beta_sigmoid ? dbt * bt * (1.f - bt) : dbt;
                b.dbeta[o] = __builtin_bit_cast(uint16_t, (__bf16)db);
                if (b.dg_act)
                    b.dg_act[o] = x;
                else
                    b.dg[o] = __builtin_bit_cast(uint16_t, (__bf16)x);
            }
        }
    }
    // through the L2 norm: dx = r dy - r^2 x (x . r dy), y = r x
    float gq[2] = {0.f, 0.f}, gk[2] = {0.f, 0.f};
    if (p.pre.qk_l2norm) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int t = 2 * half + u;
            const float a = sum_groups(dot4(row_of(L::Q, t), dq[u])), c = sum_groups(dot4(row_of(L::KM, t), dk[u]));
            if (grp == 0) {
                sc.dot[0][dims][16 * t + r] = a;
                sc.dot[1][dims][16 * t + r] = c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = 16 * (2 * half + u) + r;
#pragma unroll
            for (int w = 0; w < ND; ++w) {
                gq[u] += sc.dot[0][w][i];
                gk[u] += sc.dot[1][w][i];
            }
            gq[u] *= rq[i] * rq[i];
            gk[u] *= rk[i] * rk[i];
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int t = 2 * half + u;
        if (16 * t + r >= nv) continue;
        f32x4 x = dq[u], y = dk[u];
        if (p.pre.qk_l2norm) {
            x -= gq[u] * row_of(L::Q, t);
            y -= gk[u] * row_of(L::KM, t);
        }
        const int64_t o = ((bos + 16 * t + r) * p.H + h) * K + 16 * dims + 4 * grp;
        *(uint2 *)(b.dq + o) = __builtin_bit_cast(uint2, kda::to_bf16x4(x));
        *(uint2 *)(b.dk + o) = __builtin_bit_cast(uint2, kda::to_bf16x4(y));
    }
}

template <int K, int V>
hipError_t launch_backward(const BwdParams &b, hipStream_t st)
{
    const Params &p = b.f;
    const int64_t units = (int64_t)p.seq.N * p.HV, segs = (int64_t)p.seg.slots * p.HV;
    if (p.seg.chunks == 0) {
        chains_kernel<K, V, false><<<dim3(grid_for(units, 2)), dim3(4 * V), 0, st>>>(b);
    } else {
        bwd_ends_kernel<K, V><<<dim3(grid_for(segs, 2 * (V / 64) + K / 64)), dim3(256), 0, st>>>(b);
        bwd_join_kernel<K, V><<<dim3(grid_for(units, V / 8)), dim3(256), 0, st>>>(p);
        chains_kernel<K, V, true><<<dim3(grid_for(segs, 2)), dim3(4 * V), 0, st>>>(b);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.seq.T_total == 0) return e;
    local_kernel<K, V><<<dim3(p.seq.n_slots, p.H), dim3(8 * K), 0, st>>>(b);
    return hipGetLastError();
}

// ------------------------------------------------------------------------------------- gate

// One workgroup per value head, over all tokens in a fixed order.
__global__ __launch_bounds__(256) void gate_backward_kernel(Params p, bool f32, const float *dg_act,
                                                            void *dg, float *dA, float *ddt)
{
    __shared__ double part[2][256];
    const int j = blockIdx.x, tid = threadIdx.x;
    const int64_t end = kda::seq_eos(p.seq, p.seq.N - 1, 0);
    const float a = expf(p.pre.A_log[j]), bias = p.pre.dt_bias ? p.pre.dt_bias[j] : 0.f;
    double sa = 0.0, sb = 0.0;
    for (int64_t t = tid; t < end; t += 256) {
        const int64_t at = t * p.HV + j;
        const float x = load_io(p.g, at, f32) + bias, d = dg_act[at];
        float slope, by_a;                  // d g / d x and d g / d A_log
        if (p.pre.gate == 1) {
            slope = -a * exact_sigmoid(x);
            by_a = -a * (fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))));
        } else {
            const float y = exact_sigmoid(a * x);
            slope = p.pre.lower_bound * y * (1.f - y) * a;
            by_a = slope * x;
        }
        const float dx = d * slope;
        if (f32)
            ((float *)dg)[at] = dx;
        else
            ((uint16_t *)dg)[at] = __builtin_bit_cast(uint16_t, (__bf16)dx);
        sb += dx;
        sa += (double)d * by_a;
    }
    part[0][tid] = sa;
    part[1][tid] = sb;
    for (int n = 128; n >= 1; n >>= 1) {
        __syncthreads();
        if (tid < n) {
            part[0][tid] += part[0][tid + n];
            part[1][tid] += part[1][tid + n];
        }
    }
    if (tid == 0) {
        dA[j] = (float)part[0][0];
        if (ddt) ddt[j] = (float)part[1][0];
    }
}

hipError_t launch_gate_backward(const Params &p, bool f32, const float *dg_act, void *dg,
                                float *dA_log, float *ddt_bias, hipStream_t st)
{
    gate_backward_kernel<<<dim3(p.HV), dim3(256), 0, st>>>(p, f32, dg_act, dg, dA_log, ddt_bias);
    return hipGetLastError();
}

// --------------------------------------------------------------------------------- fp32 io

__global__ __launch_bounds__(256) void activate_decay_kernel(Params p, float *act)
{
    const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (row < p.seq.T_total * p.HV) act[row] = activate_gate(p.pre, ((const float *)p.g)[row], (int)(row % p.HV));
}

hipError_t launch_activate_decay(const Params &p, float *act, hipStream_t st)
{
    const int64_t n = p.seq.T_total * p.HV;
    if (n > 0) activate_decay_kernel<<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st>>>(p, act);
    return hipGetLastError();
}

#define GDN_INST(K, V) template hipError_t launch_backward<K, V>(const BwdParams &, hipStream_t);
GDN_INST(64, 64)
GDN_INST(64, 128)
GDN_INST(128, 64)
GDN_INST(128, 128)
#undef GDN_INST

}  // namespace gdn
