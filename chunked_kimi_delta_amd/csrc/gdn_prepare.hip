// gdn_prepare.hip -- the chunk-local half of the gated delta rule: one workgroup (4 waves) per
// (64-token chunk, value head) forms A = (I + L)^-1 and M as matrix-core operands and the row
// scales (gdn_internal.h has the formulas and the record).
//
// The Gram products K K^T and Q K^T run on the matrix core from the stored bf16 rows; the fp32
// results take the decays afterwards, each one e^{Gam_i - Gam_j} of a difference held in two
// floats (from a 64-bit cumsum), so no decay is too strong. The inverse is the forward
// substitution of the 16x16 diagonal blocks (four at once in one wave, a column per lane) and
// block forward substitution between them on the fp32 matrix core: both backward stable,
// where a product of powers of L loses digits for keys that resemble each other.
//
// Measured (K = V = 128, bf16 io): 32 heads of 21412 packed tokens 131 us for 620 MB, 16 heads x 4096 tokens
// 16 us for 58 MB: about 91% and 70% of what a large copy reaches (first calls 147 and 18 us); a workgroup alone
// takes 6 us (two to three of them in the loads, one in the diagonal blocks' substitution), and four share a
// compute unit (102 registers). First calls with Q staged in LDS next to K, also four, 184 and 18 us; with Q in
// registers, the gate's parameters loaded behind the decays, every key tile read twice and seven workgroups a
// compute unit (72 registers) 151 and 19.9 us: fewer waits did as much as more waves.
#include <type_traits>

#include "gdn_internal.h"

namespace gdn {

namespace {

// L and the inverse X in LDS: 16x16 blocks of the lower triangle, rows of 20 floats. X's diagonal blocks
// take the place of L's (the one wave that inverts them reads all of a block first).
constexpr int BP = 20, BLK = 16 * BP, BLOCKS = 16;

__device__ __forceinline__ float *block_l(float *m, int i, int j) { return m + (i * (i + 1) / 2 + j) * BLK; }
__device__ __forceinline__ float *block_x(float *m, int i, int j) {
    return i == j ? block_l(m, i, i) : m + (10 + i * (i - 1) / 2 + j) * BLK;
}
__device__ __forceinline__ f32x4 block_a(const float *b, int grp, int r) { return *(const f32x4 *)(b + r * BP + 4 * grp); }
__device__ __forceinline__ f32x4 block_b(const float *b, int grp, int r) {
    f32x4 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = b[(4 * grp + i) * BP + r];
    return x;
}
__device__ __forceinline__ void block_put(float *b, int grp, int r, f32x4 x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) b[(4 * grp + i) * BP + r] = x[i];
}

struct Scalars {                            // per token of the chunk
    float ghi[64], glo[64];                 // Gam log2(e) as the sum of two floats
    float beta[64], rk[64], rq[64];
};

// sum of the squares of eight values
template <int IN>
__device__ __forceinline__ float squares(const Parts<IN> &x) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float v = (float)x.p[0][e];
        if constexpr (IN == 3) v += (float)x.p[1][e] + (float)x.p[2][e];
        s += v * v;
    }
    return s;
}

}  // namespace

// IN: planes of q and k (1: bf16 io, 3: fp32 io); X: parts of A and M
// BWD: the backward's record (RecB).
template <int K, int IN, int X, bool BWD>
__global__ __launch_bounds__(256, IN == 3 ? 1 : 4) void prepare_kernel(Params p)
{
    constexpr int MAT = 64 * K * 2;         // bytes of one staged plane
    using R = std::conditional_t<BWD, RecB, Rec<X>>;
    constexpr int R_M = [] { if constexpr (BWD) return RecB::MT; else return Rec<X>::M; }();
    // L and X take the place of K once the Gram products are done, and each wave holds its tile of Q in
    // registers: LDS does not limit the workgroups of a compute unit (but for three planes of K = 128)
    constexpr int LX = BLOCKS * BLK * 4, AREA = IN * MAT > LX ? IN * MAT : LX;
    __shared__ __attribute__((aligned(1024))) uint8_t km[AREA];
    __shared__ Scalars sc;
    float *const lx = (float *)km;
    const int tid = threadIdx.x, lane = tid & 63, grp = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = blockIdx.x, j = blockIdx.y, h = j / p.G;
    int s, nv;
    int64_t bos;
    if (!kda::locate_slot<CT>(p.seq, slot, &s, &bos, &nv)) return;

    // every load at once: what one wave needs for the scalars first (loads complete in order)
    const bool live = lane < nv;
    float g = 0.f, b = 0.f;
    const GateHead gate = gate_head(p.pre, j);
    if (wave == 0) {
        const int64_t at = (bos + (live ? lane : nv - 1)) * p.HV + j;
        g = load_io(p.g, at, IN == 3);
        b = load_io(p.beta, at, IN == 3);
    }
    const int64_t stride = (int64_t)p.H * K, off = (bos * p.H + h) * K;
    const int ti = 3 - wave, qi = 16 * ti + r;          // the wave's query tile, the lane's row of it
    Parts<IN> qt[K / 32];
#pragma unroll
    for (int i = 0; i < IN; ++i) {
        const uint16_t *const q = p.q[i] + off + (qi < nv ? qi : nv - 1) * stride + 8 * grp;
#pragma unroll
        for (int st = 0; st < K / 32; ++st) qt[st].p[i] = *(const bf16x8 *)(q + 32 * st);
        stage_rows<K, 4>(p.k[i] + off, stride, nv, km + i * MAT, wave, lane);
    }
    kda::vm_drain();
    __syncthreads();
    if (wave == 0) {
        g = activate_gate(p.pre, g, gate);
        if (p.pre.beta_sigmoid) b = exact_sigmoid(b);
        // a decay below e^-100000 is zero whatever its size; -inf would make differences NaN
        if (g < -1e5f) g = -1e5f;
        double x = live ? (double)g * 1.4426950408889634 : 0.0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double y = __shfl_up(x, d);
            if (lane >= d) x += y;
        }
        const float hi = (float)x;
        sc.ghi[lane] = hi;
        sc.glo[lane] = (float)(x - (double)hi);
        sc.beta[lane] = live ? b : 0.f;
    } else if (wave < 3) {                  // meanwhile: two neighbouring threads a row of K
        const int row = (tid - 64) >> 1, part = tid & 1;
        float f = 1.f;
        if (p.pre.qk_l2norm) {
            f = 0.f;
#pragma unroll
            for (int c = 0; c < K / 16; ++c) f += squares(lds_parts<IN>(km + piece_at<K>(row, part * (K / 16) + c), MAT));
            f += __shfl_xor(f, 1);
            f = 1.f / sqrtf(f + kda::L2NORM_EPS);
        }
        if (part == 0) sc.rk[row] = f;
    }
    {
        float f = 1.f;
        if (p.pre.qk_l2norm) {
            f = 0.f;
#pragma unroll
            for (int c = 0; c < K / 32; ++c) f += squares(qt[c]);
            f = 1.f / sqrtf(sum_groups(f) + kda::L2NORM_EPS);
        }
        if (grp == 0) sc.rq[qi] = f;
    }
    __syncthreads();

    uint8_t *const rec = p.rec + ((size_t)j * p.seq.n_slots + slot) * R::BYTES;
    auto k_tile = [&](int t, int st) { return lds_parts<IN>(km + piece_at<K>(16 * t + r, 4 * st + grp), MAT); };
    auto four = [&](const float *x, int t) { return *(const f32x4 *)(x + 16 * t + 4 * grp); };
    // e^{Gam_i - Gam_j}, the exponents held in two floats each
    auto decay = [&](float hi, float lo) { return __builtin_amdgcn_exp2f(hi + lo); };
    // L's row tile `wave` and M's query tile 3 - wave, five tiles a wave. A lane's four values are
    // consecutive columns j of a row i (in the backward's M, which is stored transposed, consecutive rows
    // of a column); a key tile serves both.
    const int li = 16 * wave + r;
    Parts<IN> kt[K / 32];
#pragma unroll
    for (int st = 0; st < K / 32; ++st) kt[st] = k_tile(wave, st);
    const float lhi = sc.ghi[li], llo = sc.glo[li], lrk = sc.rk[li];
    const f32x4 mhi = BWD ? four(sc.ghi, ti) : f32x4{sc.ghi[qi]}, mlo = BWD ? four(sc.glo, ti) : f32x4{sc.glo[qi]};
    f32x4 mrq = BWD ? four(sc.rq, ti) : f32x4{sc.rq[qi]};
    mrq *= p.scale;
    f32x4 lt[4];
#pragma unroll
    for (int tj = 0; tj < 4; ++tj) {
        lt[tj] = zero4();
        if (tj > wave && tj > (ti | 1)) continue;
        Parts<IN> x[K / 32];
#pragma unroll
        for (int st = 0; st < K / 32; ++st) x[st] = k_tile(tj, st);
        const f32x4 hi = four(sc.ghi, tj), lo = four(sc.glo, tj), s = four(sc.rk, tj) * four(sc.beta, tj);
        const int j0 = 16 * tj + 4 * grp;
        if (tj <= wave) {
            f32x4 c = zero4();
#pragma unroll
            for (int st = 0; st < K / 32; ++st) c = mm(x[st], kt[st], c);
#pragma unroll
            for (int e = 0; e < 4; ++e) lt[tj][e] = li > j0 + e ? c[e] * (lrk * s[e]) * decay(lhi - hi[e], llo - lo[e]) : 0.f;
        }
        if (tj > (ti | 1)) continue;
        f32x4 m = zero4();
        if (tj <= ti) {
            f32x4 c = zero4();
            if constexpr (BWD) {
                const int jj = 16 * tj + r;
                const float ch = sc.ghi[jj], cl = sc.glo[jj], cs = sc.rk[jj] * sc.beta[jj];
#pragma unroll
                for (int st = 0; st < K / 32; ++st) c = mm(qt[st], x[st], c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 16 * ti + 4 * grp + e;
                    m[e] = i >= jj && i < nv ? c[e] * (mrq[e] * cs) * decay(mhi[e] - ch, mlo[e] - cl) : 0.f;
                }
            } else {
#pragma unroll
                for (int st = 0; st < K / 32; ++st) c = mm(x[st], qt[st], c);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    m[e] = qi >= j0 + e && qi < nv ? c[e] * (mrq[0] * s[e]) * decay(mhi[0] - hi[e], mlo[0] - lo[e]) : 0.f;
            }
        }
        uint8_t *at = rec + lane * 16 + (BWD ? R_M + frag_index_t(tj, ti >> 1) * R::FR + (ti & 1) * 8
                                             : R_M + frag_index(ti, tj >> 1) * R::FR + (tj & 1) * 8);
#pragma unroll
        for (int k = 0; k < X; ++k) {
            const kda::bf16x4 y = kda::to_bf16x4(m);
            *(uint2 *)(at + k * R::MAT) = __builtin_bit_cast(uint2, y);
#pragma unroll
            for (int e = 0; e < 4; ++e) m[e] -= (float)y[e];
        }
    }
    __syncthreads();
#pragma unroll
    for (int tj = 0; tj < 4; ++tj)
        if (tj <= wave) *(f32x4 *)(block_l(lx, wave, tj) + r * BP + 4 * grp) = lt[tj];
    __syncthreads();
    if (wave == 0) {                        // the four diagonal blocks, column r of block grp
        float x[16];
        float *const m = block_l(lx, grp, grp);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float acc = i == r ? 1.f : 0.f;
#pragma unroll
            for (int jj = 0; jj < i; ++jj) acc -= m[i * BP + jj] * x[jj];
            x[i] = acc;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) m[i * BP + r] = x[i];
    }
    __syncthreads();
    auto l_a = [&](int bi, int bj) { return block_a(block_l(lx, bi, bj), grp, r); };
    auto x_a = [&](int bi, int bj) { return block_a(block_x(lx, bi, bj), grp, r); };
    auto x_b = [&](int bi, int bj) { return block_b(block_x(lx, bi, bj), grp, r); };
    auto neg = [](f32x4 x) { return f32x4{-x[0], -x[1], -x[2], -x[3]}; };
    if (wave < 2) {                         // X_10 = -X_11 L_10 X_00, X_32 = -X_33 L_32 X_22
        const int lo = 2 * wave, hi = lo + 1;
        const f32x4 t = kda::mm16_f32(l_a(hi, lo), x_b(lo, lo), zero4());
        block_put(block_x(lx, hi, lo), grp, r, neg(kda::mm16_f32(x_a(hi, hi), t, zero4())));
    }
    __syncthreads();
    {                                       // X_ij = -sum_k X_ik (L X)_kj, i = 2, 3, j = 0, 1
        const int i = 2 + (wave >> 1), c = wave & 1;
        auto row_of = [&](int row) {        // (L X) of block row `row`, block column c
            f32x4 t = kda::mm16_f32(l_a(row, c), x_b(c, c), zero4());
            return c == 0 ? kda::mm16_f32(l_a(row, 1), x_b(1, 0), t) : t;
        };
        const f32x4 t2 = row_of(2);
        f32x4 x = kda::mm16_f32(x_a(i, 2), t2, zero4());
        if (i == 3) x = kda::mm16_f32(x_a(3, 3), row_of(3), x);
        block_put(block_x(lx, i, c), grp, r, neg(x));
    }
    __syncthreads();
    for (int f = wave; f < 6; f += 4) {     // A's fragments
        const int t = f < 2 ? f : 2 + ((f - 2) >> 1), st = f < 2 ? 0 : (f & 1);
        f32x4 x[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int bj = 2 * st + u;
            x[u] = bj <= t ? x_a(t, bj) : zero4();
            if (bj == t)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[u][e] = 4 * grp + e <= r ? x[u][e] : 0.f;
        }
        const Parts<X> y = split<X>(x[0], x[1]);
        const auto rs = kda::buffer_rsrc(rec, R::BYTES);
#pragma unroll
        for (int k = 0; k < X; ++k)
            kda::bstore16<0>(rs, f * R::FR + lane * 16, R::A + k * R::MAT, y.p[k]);
    }
    if constexpr (BWD) {
        for (int f = wave; f < 6; f += 4) { // A^T's fragments
            const int t = f < 4 ? f >> 1 : f - 2, st = f < 4 ? (f & 1) : 1;
            f32x4 x[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int bi = 2 * st + u;
                x[u] = bi >= t ? x_b(bi, t) : zero4();
                if (bi == t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[u][e] = 4 * grp + e >= r ? x[u][e] : 0.f;
            }
            const Parts<X> y = split<X>(x[0], x[1]);
            const auto rs = kda::buffer_rsrc(rec, R::BYTES);
#pragma unroll
            for (int k = 0; k < X; ++k)
                kda::bstore16<0>(rs, f * R::FR + lane * 16, R::AT + k * R::MAT, y.p[k]);
        }
        if (wave == 2) {
            ((float *)(rec + R::GHI))[lane] = sc.ghi[lane];
            ((float *)(rec + R::GLO))[lane] = sc.glo[lane];
            ((float *)(rec + R::BETA))[lane] = sc.beta[lane];
            ((float *)(rec + R::RK))[lane] = sc.rk[lane];
            ((float *)(rec + R::RQ))[lane] = sc.rq[lane];
        }
    }
    if (wave == 3) {
        const float whi = sc.ghi[63], wlo = sc.glo[63];
        const float head = __builtin_amdgcn_exp2f(sc.ghi[lane] + sc.glo[lane]);
        const float tail = __builtin_amdgcn_exp2f((whi - sc.ghi[lane]) + (wlo - sc.glo[lane]));
        ((float *)(rec + R::RA))[lane] = head * sc.rk[lane];
        ((float *)(rec + R::RB))[lane] = tail * sc.rk[lane] * sc.beta[lane];
        ((float *)(rec + R::RC))[lane] = lane < nv ? p.scale * head * sc.rq[lane] : 0.f;
        ((float *)(rec + R::EG))[lane] = __builtin_amdgcn_exp2f(whi + wlo);
    }
}

// fp32 q and k (blockIdx.y) as three bf16 planes each: their sum is x to 2^-24 or better
__global__ __launch_bounds__(256) void split_planes_kernel(const float *q, const float *k, int64_t n4,
                                                           uint2 *q_planes, uint2 *k_planes)
{
    const float *const x = blockIdx.y ? k : q;
    uint2 *const planes = blockIdx.y ? k_planes : q_planes;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n4) return;
    f32x4 v = ((const f32x4 *)x)[i];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const kda::bf16x4 y = kda::to_bf16x4(v);
        planes[j * n4 + i] = __builtin_bit_cast(uint2, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] -= (float)y[e];
    }
}

hipError_t launch_split_planes(const float *q, const float *k, int64_t n, uint16_t *q_planes, uint16_t *k_planes,
                               hipStream_t st)
{
    const int64_t n4 = n / 4;               // rows are 64 or 128 wide
    if (n4 == 0) return hipSuccess;
    split_planes_kernel<<<dim3((unsigned)((n4 + 255) / 256), 2), dim3(256), 0, st>>>(q, k, n4, (uint2 *)q_planes,
                                                                                     (uint2 *)k_planes);
    return hipGetLastError();
}

template <int K>
hipError_t launch_prepare(const Params &p, bool f32, hipStream_t st)
{
    const dim3 grid(p.seq.n_slots, p.HV);
    if (f32)
        prepare_kernel<K, 3, 3, false><<<grid, dim3(256), 0, st>>>(p);
    else
        prepare_kernel<K, 1, 2, false><<<grid, dim3(256), 0, st>>>(p);
    return hipGetLastError();
}

template <int K>
hipError_t launch_prepare_bwd(const Params &p, hipStream_t st)
{
    prepare_kernel<K, 1, 2, true><<<dim3(p.seq.n_slots, p.HV), dim3(256), 0, st>>>(p);
    return hipGetLastError();
}

template hipError_t launch_prepare_bwd<64>(const Params &, hipStream_t);
template hipError_t launch_prepare_bwd<128>(const Params &, hipStream_t);
template hipError_t launch_prepare<64>(const Params &, bool, hipStream_t);
template hipError_t launch_prepare<128>(const Params &, bool, hipStream_t);

}  // namespace gdn
