// gdn_internal.h -- device-side building blocks of the gated delta rule (one decay per token
// and value head) on gfx950. Lane layouts are those of kda_internal.h.
//
// A sequence is cut into chunks of 64 tokens (four 16-token tiles). With Gam the in-chunk
// cumsum of g, gam its last value, D_ij = e^{Gam_i - Gam_j} and S the state at the chunk's
// start, a chunk is
//     R = V - e^Gam . (K S)                         e = A R,  A = (I + L)^-1,
//     o = scale e^Gam . (Q S) + M e                 L_ij = D_ij beta_j k_i.k_j   (i > j)
//     S <- e^gam S + K^T (beta e^{gam - Gam} . e)   M_ij = scale D_ij beta_j q_i.k_j  (i >= j)
// where e_t is the residual v_t - S_{t-1}^T k_t of the token recurrence itself (beta enters
// after it). With one decay per token every decay is a scalar of a row: K, Q and V enter the
// matrix products as they are stored, and the decays, beta and the L2-norm factors are row
// scales of the products' results.
//
// Operands with more than 8 significant bits (S, R, e, A, M, fp32 inputs) are split into bf16
// parts, x = x0 + x1 (+ x2), and a product takes the pairs i + j < parts: two parts hold 17 bits
// (bf16 io), three hold 24 (fp32 io, whose q and k come as three planes). So an fp32 state is an
// fp32-class result for either io type.
#pragma once

#include "kda_internal.h"

namespace gdn {

using kda::bf16x8;
using kda::f32x4;
using kda::mfma32;
using kda::SeqGeom;
using kda::zero4;

constexpr int CT = 64;                  // tokens per chunk

// Segments of `chunks` chunks each, where a batch is too small to fill the device (chunks > 0). Segment
// i of sequence s lies in slot floor(bos_s / (64 chunks)) + s + i. A chunk step is affine in the state,
// so with PHI_i the transition of segment i (its end state from the identity, without v) and E_i its end
// state from zero (segment 0: from the initial state), the true end states are
//     E_i <- PHI_i E_{i-1} + E_i,
// and in reverse the gradients before the segments G_i <- PHI_i^T G_{i+1} + G_i, G_i from zero (the last
// segment: from dht). First pass: E, G and PHI of all segments side by side; the few products above; then
// every segment from its true start. The last segment's slot of E is not needed
// for that and holds a copy of the initial state (which final_state may overwrite); the first one's of G is unused.
struct Segments {
    int32_t chunks, slots;
    float *E, *G, *PHI;                 // [slots][HV][K][V], the same, [slots][HV][2][K][K] (and transposed)
};

struct Pre {
    int32_t qk_l2norm, beta_sigmoid, gate;
    float lower_bound;
    const float *A_log, *dt_bias;       // [HV] (dt_bias may be null)
};

struct Params {
    SeqGeom seq;                        // n_slots counts 64-token chunk slots
    int32_t H, HV, G;
    float scale;
    const uint16_t *q[3], *k[3];        // bf16 io: q and k; fp32 io: their three bf16 planes
    const void *v, *g, *beta;           // io dtype
    const float *h0;
    void *o;                            // io dtype
    float *ht;
    uint8_t *rec;                       // chunk records
    Pre pre;
    Segments seg;
};

struct BwdParams {
    Params f;                           // f.rec: RecB records
    const uint16_t *d_o;                // [T_total][HV][V]
    const float *dht;                   // or null (zero)
    uint8_t *keep;                      // Keep records
    uint16_t *dq, *dk, *dv;             // bf16, like q, k, v
    uint16_t *dbeta, *dg;               // [T_total][HV] (dg: no gate)
    float *dg_act;                      // [T_total][HV] gradient of the activated decay (gate)
    float *dh0;                         // or null
};

// Arguments of the recurrence (gdn_step, and gdn_fwd for short dense batches).
struct StepParams {
    int32_t B, T, H, HV, G;
    float scale;
    const void *q, *k, *v, *g, *beta;
    void *o;
    const float *h0;                    // row b's state: h0 / ht at index[b] (or b)
    float *ht;
    const int32_t *index;
    int32_t slots;
    Pre pre;
};

// Record of one (value head, chunk slot). A and M are lower triangular; their 16-row tiles t
// are stored as 16x16x32 operand fragments over the tokens 32 s .. 32 s + 31, s <= t / 2, in
// the order (0,0) (1,0) (2,0) (2,1) (3,0) (3,1): lane (g, m) holds row 16 t + m, elements e < 4
// token 32 s + 4 g + e and e >= 4 token 32 s + 16 + 4 g + e - 4 (so that two C-layout tiles are
// the other operand, as they are).
//   A and M, each [parts][6][64 lanes][8] bf16; between them fp32 row scales of the 64 tokens:
//   RA = e^Gam rk, RB = beta e^{gam - Gam} rk, RC = scale e^Gam rq (rk, rq the L2-norm factors),
//   and EG [1] = e^gam. Copied to LDS in 1 KiB steps, without M where there is no output.
template <int X>
struct Rec {
    static constexpr int FR = 1024, MAT = 6 * FR;       // one fragment, one part of a matrix
    static constexpr int A = 0;
    static constexpr int RA = X * MAT, RB = RA + 256, RC = RB + 256, EG = RC + 256;
    static constexpr int M = RA + FR;
    static constexpr int BYTES = M + X * MAT;
};

__host__ __device__ constexpr int frag_index(int t, int s) { return t < 2 ? t : 2 * t - 2 + s; }

// Record of the backward (bf16 io, two parts): A as above and the row scales, then A^T and M^T,
// upper triangular, tile t over the tokens of s >= t / 2 in the order (0,0) (0,1) (1,0) (1,1)
// (2,1) (3,1), and more scalars per token: Gam log2(e) in two floats, beta, rk, rq.
struct RecB {
    static constexpr int X = 2, FR = 1024, MAT = 6 * FR;
    static constexpr int A = 0, RA = X * MAT, RB = RA + 256, RC = RB + 256, EG = RC + 256;
    static constexpr int AT = RA + FR, MT = AT + X * MAT;
    static constexpr int GHI = MT + X * MAT, GLO = GHI + 256, BETA = GLO + 256, RK = BETA + 256,
                         RQ = RK + 256;
    static constexpr int BYTES = GHI + 2 * FR;
    static constexpr int REV = RA, REV_KIB = 1 + 2 * X * 6;     // what the reverse pass reads
};

__host__ __device__ constexpr int frag_index_t(int t, int s) { return t < 2 ? 2 * t + s : 2 + t; }

// What the backward's two passes leave for one (value head, chunk slot), fp16 with a power of two
// for each of the two states and for each token of e and dR (16-bit values of 11 significant bits: the
// products that use them then add little to the rounding of a bf16 gradient): the state at the chunk's start
// and the gradient of the state at its end, e, and the gradient of R (which is v's); then the factors that
// undo the scales, fp32: the two states', from SE on the 64 tokens' of e, from SR on of dR. What lies 2^-28
// and more below the largest value of its state or its token's row has fewer bits. Stored in blocks of 16 columns, as a wave of the passes holds them (a
// lane: consecutive key dims or tokens of one column), so that it stores whole lines:
//   S, DS [V/16][K/32][16 columns][32 key dims],  E, DR [V/16][4][16 columns][16 tokens].
template <int K, int V>
struct Keep {
    static constexpr int S = 0, DS = V * K * 2, E = 2 * DS, DR = E + V * 128, SCALE = DR + V * 128;
    static constexpr int SE = 64, SR = 128, BYTES = SCALE + 1024;   // (copied to LDS as one KiB)
    // bytes to four key dims from `dim`, or four tokens from `tok`, of column `col`
    static __host__ __device__ constexpr int state_at(int col, int dim) {
        return ((col >> 4) * (K / 32) + (dim >> 5)) * 1024 + (col & 15) * 64 + (dim & 31) * 2;
    }
    static __host__ __device__ constexpr int row_at(int col, int tok) {
        return ((col >> 4) * 4 + (tok >> 4)) * 512 + (col & 15) * 32 + (tok & 15) * 2;
    }
};

// ------------------------------------------------------------------------------- operands

template <int X>
struct Parts {
    bf16x8 p[X];
};

// Eight values (two C-layout tiles) as X bf16 parts. Two values are rounded by one instruction and
// their rounded parts taken back from the packed pair: three instructions a value for two parts.
template <int X>
__device__ __forceinline__ Parts<X> split(f32x4 x, f32x4 y) {
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
    Parts<X> r;
    float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
    for (int k = 0; k < X; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(kda::f32v2{v[2 * i], v[2 * i + 1]}, bf16x2));
            if (k + 1 < X) {
                v[2 * i] -= kda::bf16lo(w[i]);
                v[2 * i + 1] -= kda::bf16hi(w[i]);
            }
        }
        r.p[k] = __builtin_bit_cast(bf16x8, kda::u32x4{w[0], w[1], w[2], w[3]});
    }
    return r;
}

template <int XA, int XB>
__device__ __forceinline__ f32x4 mm(const Parts<XA> &a, const Parts<XB> &b, f32x4 c) {
    constexpr int X = XA > XB ? XA : XB;
#pragma unroll
    for (int i = 0; i < XA; ++i)
#pragma unroll
        for (int j = 0; j < XB; ++j)
            if (i + j < X) c = mfma32(a.p[i], b.p[j], c);
    return c;
}

// ---------------------------------------------------------------------- scaled 16-bit values

// The largest of a wave's values (every lane gets it); x >= 0, NaN and infinities included.
__device__ __forceinline__ float wave_max(float x) {
    uint32_t u = __float_as_uint(x);
    auto step = [&](uint32_t y) { u = u > y ? u : y; };
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x111, 0xf, 0xf, false));  // row_shr:1
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x112, 0xf, 0xf, false));
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x114, 0xf, 0xf, false));
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x118, 0xf, 0xf, false));
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x142, 0xa, 0xf, false));  // row_bcast:15
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x143, 0xc, 0xf, false));  // row_bcast:31
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)u, 63));
}

// Sum over the four lanes that share lane % 16 (every one gets it): two exchanges of half a wave and of
// neighbouring rows of 16 lanes, without LDS.
__device__ __forceinline__ float sum_groups(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto c = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(c[0]) + __uint_as_float(c[1]);
}

__device__ __forceinline__ float max_abs(f32x4 x, float m) {
    return fmaxf(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))), m);
}

// The power of two that brings values of magnitude up to `most` to just below 2^14 (fp16 then has
// 11 bits for everything down to 2^-28 of the largest), and its inverse. Below 2^-113 the inverse
// is clamped: such values turn subnormal.
struct Scale {
    float f, inv;
};
__device__ __forceinline__ Scale scale_for(float most) {
    const uint32_t e0 = __float_as_uint(most) >> 23, e = e0 < 14 ? 14 : e0;
    return Scale{__uint_as_float((267u - e) << 23), __uint_as_float((e - 13u) << 23)};
}

__device__ __forceinline__ uint2 half4(f32x4 x, float f) {
    return __builtin_bit_cast(uint2, kda::to_f16x4(x * f));
}

typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((ext_vector_type(4))) short s16x4;

__device__ __forceinline__ bf16x8 lds_b128(const uint8_t *p) { return *(const bf16x8 *)p; }
// the parts of an operand, `step` bytes apart
template <int X>
__device__ __forceinline__ Parts<X> lds_parts(const uint8_t *p, int step) {
    Parts<X> r;
#pragma unroll
    for (int i = 0; i < X; ++i) r.p[i] = lds_b128(p + i * step);
    return r;
}

// Transposing read: within 16 lanes, lane j reads four 16-bit values of row j / 4 at its own
// address and lane m receives column m of rows 0 .. 3 (m = 4 (j % 4) + element).
__device__ __forceinline__ s16x4 lds_tr(const uint8_t *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4 *)(lds_u8 *)p);
}
__device__ __forceinline__ bf16x8 join(s16x4 a, s16x4 b) {
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ __forceinline__ f32x4 widen(s16x4 a) {
    f32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __uint_as_float((uint32_t)(uint16_t)a[i] << 16);
    return r;
}

// A staged matrix has rows of W 16-bit values in 16-byte pieces; piece p of row r lies at place
// p ^ swizzle(r) of its row. Sixteen lanes of a transposing read take four neighbouring rows of two
// or four pieces, sixteen lanes of a 16-byte read one piece of sixteen rows: the two low bits of the
// row spread the former over the banks (a row of 64 values fills only half of them, so there the
// lowest bit does without), the next two the latter. Against p ^ (r % 16) the first pass over segments loses 38
// instead of 47% of its LDS cycles to bank conflicts, the state pass as many (37 and 36%): gradients of 16 heads x
// 4096 tokens 220 -> 216 us, the forward as fast.
template <int W>
__device__ __forceinline__ int swizzle(int row) {
    return W == 128 ? (row & 3) << 2 | (row >> 2 & 3) : (row & 2) << 1 | (row >> 2 & 3);
}
template <int W>
__device__ __forceinline__ int piece_at(int row, int piece) {
    constexpr int NP = W / 8;
    return (row * NP + (piece ^ swizzle<W>(row))) * 16;
}

// 16 bytes per lane, from base + off, to LDS at dst + 16 lane (base and dst uniform). Written out,
// because behind the builtin the compiler waits for every copy in flight before the next transposing
// read of LDS, also where the copies go to the other buffer. The kernels wait themselves (vm_drain)
// before the barrier behind which the data is read. M0 takes its value one cycle before the copy
// reads it (s_nop).
// (The compiler keeps M0 for itself and warns of the clobber, which is what tells it of the write.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16_to_lds(const void *base, uint32_t off, uint8_t *dst) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_u8 *)dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(at), "v"(off), "s"(base) : "memory", "m0");
}
#pragma clang diagnostic pop

// Stages 64 rows of W 16-bit values (rows `stride` values apart) into LDS, layout piece_at, NW waves
// sharing the work. A wave's steps are NW * (64 / pieces) rows apart, a multiple of the rows after
// which the swizzle repeats, so one offset per lane serves them all. Rows from nv on repeat row
// nv - 1: every read lies inside the sequence, and the row scales and operands that meet such rows are
// zero. No wait.
template <int W, int NW>
struct RowStage {
    static constexpr int NP = W / 8, ROWS = 64 / NP, STEPS = NP / NW;
    static_assert(STEPS >= 1 && (STEPS == 1 || NW * ROWS % (W == 128 ? 16 : 8) == 0), "one offset per lane");
    int row, piece;
    uint32_t off;                           // bytes
    int64_t stride;
    __device__ __forceinline__ RowStage(int64_t stride_, int wave, int lane) : stride(stride_) {
        row = wave * ROWS + lane / NP;
        piece = (lane % NP) ^ swizzle<W>(row);
        off = (uint32_t)((row * stride + piece * 8) * 2);
    }
    __device__ __forceinline__ void operator()(const uint16_t *src, int nv, uint8_t *dst, int wave) const {
#pragma unroll
        for (int q = 0; q < STEPS; ++q) {
            uint8_t *const to = dst + (q * NW + wave) * 1024;
            if (nv == 64) {
                copy16_to_lds(src + q * NW * ROWS * stride, off, to);
            } else {
                const int r = row + q * NW * ROWS;
                copy16_to_lds(src, (uint32_t)(((r < nv ? r : nv - 1) * stride + piece * 8) * 2), to);
            }
        }
    }
};

template <int W, int NW>
__device__ __forceinline__ void stage_rows(const uint16_t *src, int64_t stride, int nv, uint8_t *dst, int wave,
                                           int lane) {
    RowStage<W, NW>(stride, wave, lane)(src, nv, dst, wave);
}

// Stage `KIB` KiB of consecutive memory.
template <int KIB, int NW>
__device__ __forceinline__ void stage_block(const uint8_t *src, uint8_t *dst, int wave, int lane) {
#pragma unroll
    for (int q = 0; q < (KIB + NW - 1) / NW; ++q) {
        const int step = q * NW + wave;
        if (step < KIB) copy16_to_lds(src + step * 1024, lane * 16, dst + step * 1024);
    }
}

// ------------------------------------------------------------------------------- pre-stage

__device__ __forceinline__ float exact_sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// A head's gate parameters, loaded ahead of their use.
struct GateHead {
    float A_log, bias;
};
__device__ __forceinline__ GateHead gate_head(const Pre &pre, int j) {
    GateHead h = {0.f, 0.f};
    if (pre.gate) {
        h.A_log = pre.A_log[j];
        if (pre.dt_bias) h.bias = pre.dt_bias[j];
    }
    return h;
}

// The log decay of raw input x (bias not added yet).
__device__ __forceinline__ float activate_gate(const Pre &pre, float x, GateHead h) {
    if (pre.gate == 0) return x;
    x += h.bias;
    const float a = expf(h.A_log);
    if (pre.gate == 1) return -a * (fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))));
    return pre.lower_bound * exact_sigmoid(a * x);
}
__device__ __forceinline__ float activate_gate(const Pre &pre, float x, int j) {
    return activate_gate(pre, x, gate_head(pre, j));
}

__device__ __forceinline__ float load_io(const void *p, int64_t i, bool f32) {
    return f32 ? ((const float *)p)[i] : kda::bf16_bits_to_f32(((const uint16_t *)p)[i]);
}

}  // namespace gdn

// Host-side launchers (defined next to their kernels).
namespace gdn {
// fp32 q and k [n] as three bf16 planes each, n values apart
hipError_t launch_split_planes(const float *q, const float *k, int64_t n, uint16_t *q_planes, uint16_t *k_planes,
                               hipStream_t st);
template <int K> hipError_t launch_prepare(const Params &p, bool f32, hipStream_t st);
template <int K> hipError_t launch_prepare_bwd(const Params &p, hipStream_t st);    // bf16 io
template <int K, int V> hipError_t launch_backward(const BwdParams &b, hipStream_t st);
// The gate's share of the backward: dg and (summed over all tokens of all sequences) dA_log and
// ddt_bias (or null) from the gradient of the activated decay.
hipError_t launch_gate_backward(const Params &p, bool f32, const float *dg_act, void *dg,
                                float *dA_log, float *ddt_bias, hipStream_t st);
// Rows of 8-bit checkpoints (include/act8.h) back in the io type: three tensors, one launch.
hipError_t launch_unpack3(const int8_t *const data[3], const float *const scale[3], const int64_t rows[3],
                          const int32_t D[3], void *const x[3], bool f32, hipStream_t st);
// fp32 io: the activated decay [T_total][HV]
hipError_t launch_activate_decay(const Params &p, float *act, hipStream_t st);
template <int K, int V> hipError_t launch_state(const Params &p, bool f32, hipStream_t st);
template <int K, int V> hipError_t launch_recurrent(const StepParams &p, bool f32, hipStream_t st);
}  // namespace gdn
