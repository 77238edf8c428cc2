// gdn_prepare.hip -- the chunk-local half of the gated delta rule: one workgroup (4 waves) per
// (64-token chunk, value head) forms A = (I + L)^-1 and M as matrix-core operands and the row
// scales (gdn_internal.h has the formulas and the record).
//
// The Gram products K K^T and Q K^T run on the matrix core from the stored bf16 rows; the fp32
// results take the decays afterwards, each one e^{Gam_i - Gam_j} of a difference held in two
// floats (from a 64-bit cumsum), so no decay is too strong. The inverse is the forward
// substitution of the 16x16 diagonal blocks (four at once in one wave, a column per lane) and
// block forward substitution between them on the fp32 matrix core: both backward stable, where
// a product of powers of L loses digits for keys that resemble each other.
#include <type_traits>

#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int P = 68;                       // floats per row of a 64 x 64 matrix in LDS

__device__ __forceinline__ f32x4 block_a(const float *m, int bi, int bj, int grp, int r) {
    return *(const f32x4 *)(m + (16 * bi + r) * P + 16 * bj + 4 * grp);
}
__device__ __forceinline__ f32x4 block_b(const float *m, int bi, int bj, int grp, int r) {
    f32x4 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = m[(16 * bi + 4 * grp + i) * P + 16 * bj + r];
    return x;
}
__device__ __forceinline__ void block_put(float *m, int bi, int bj, int grp, int r, f32x4 x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m[(16 * bi + 4 * grp + i) * P + 16 * bj + r] = x[i];
}

struct Scalars {                            // per token of the chunk
    float ghi[64], glo[64];                 // Gam log2(e) as the sum of two floats
    float beta[64], rk[64], rq[64];
};

// 1 / sqrt(sum of squares + 1e-6) of a staged row, its quarter `part` per thread (four threads
// of a row are neighbours)
template <int K, int IN>
__device__ __forceinline__ float row_factor(const uint8_t *m, int row, int part) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < K / 32; ++c) {
        const Parts<IN> x = lds_parts<IN>(m + piece_at<K>(row, part * (K / 32) + c), 64 * K * 2);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = (float)x.p[0][e];
            if constexpr (IN == 3) v += (float)x.p[1][e] + (float)x.p[2][e];
            s += v * v;
        }
    }
    s += __shfl_xor(s, 1);
    s += __shfl_xor(s, 2);
    return 1.f / sqrtf(s + kda::L2NORM_EPS);
}

}  // namespace

// IN: planes of q and k (1: bf16 io, 3: fp32 io); X: parts of A and M
// BWD: the backward's record (RecB).
template <int K, int IN, int X, bool BWD>
__global__ __launch_bounds__(256) void prepare_kernel(Params p)
{
    constexpr int MAT = 64 * K * 2;         // bytes of one staged plane
    using R = std::conditional_t<BWD, RecB, Rec<X>>;
    // L and X take the place of K and Q once the Gram products are done: with less LDS more
    // workgroups share a compute unit, which is what hides the phases' latencies
    constexpr int LX = 2 * 64 * P * 4, AREA = 2 * IN * MAT > LX ? 2 * IN * MAT : LX;
    __shared__ __attribute__((aligned(1024))) uint8_t kq[AREA];
    __shared__ Scalars sc;
    float *const Lm = (float *)kq, *const Xm = Lm + 64 * P;
    uint8_t *const km = kq, *const qm = kq + IN * MAT;
    const int tid = threadIdx.x, lane = tid & 63, grp = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = blockIdx.x, j = blockIdx.y, h = j / p.G;
    int s, nv;
    int64_t bos;
    if (!kda::locate_slot<CT>(p.seq, slot, &s, &bos, &nv)) return;

    const int64_t stride = (int64_t)p.H * K, off = (bos * p.H + h) * K;
#pragma unroll
    for (int i = 0; i < IN; ++i) {
        stage_rows<K, 4>(p.k[i] + off, stride, nv, km + i * MAT, wave, lane);
        stage_rows<K, 4>(p.q[i] + off, stride, nv, qm + i * MAT, wave, lane);
    }
    if (wave == 0) {
        const bool live = lane < nv;
        const int64_t at = (bos + (live ? lane : nv - 1)) * p.HV + j;
        float g = activate_gate(p.pre, load_io(p.g, at, IN == 3), j);
        float b = load_io(p.beta, at, IN == 3);
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
    }
    kda::vm_drain();
    __syncthreads();
    {
        const int row = tid >> 2, part = tid & 3;
        float fk = 1.f, fq = 1.f;
        if (p.pre.qk_l2norm) {
            fk = row_factor<K, IN>(km, row, part);
            fq = row_factor<K, IN>(qm, row, part);
        }
        if (part == 0) {
            sc.rk[row] = fk;
            sc.rq[row] = fq;
        }
    }
    __syncthreads();

    uint8_t *const rec = p.rec + ((size_t)j * p.seq.n_slots + slot) * R::BYTES;
    auto decay = [&](int i, int jj) {       // e^{Gam_i - Gam_jj}
        return __builtin_amdgcn_exp2f((sc.ghi[i] - sc.ghi[jj]) + (sc.glo[i] - sc.glo[jj]));
    };
    // products of row tile a of X and row tile b of Y over the K columns
    auto gram = [&](const uint8_t *x, int a, const uint8_t *y, int b) {
        f32x4 c = zero4();
#pragma unroll
        for (int st = 0; st < K / 32; ++st)
            c = mm(lds_parts<IN>(x + piece_at<K>(16 * a + r, 4 * st + grp), MAT),
                   lds_parts<IN>(y + piece_at<K>(16 * b + r, 4 * st + grp), MAT), c);
        return c;
    };
    // L row tile `wave` (rows in C-layout), and M of query tile 3 - wave, transposed, so that
    // a lane's four values are consecutive tokens of one query row: five tiles a wave
    f32x4 lt[4];
#pragma unroll
    for (int tj = 0; tj < 4; ++tj) {
        lt[tj] = zero4();
        if (tj > wave) continue;
        const f32x4 c = gram(km, wave, km, tj);
        const int jj = 16 * tj + r;
        const float sj = sc.rk[jj] * sc.beta[jj];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 16 * wave + 4 * grp + e;
            lt[tj][e] = i > jj ? c[e] * sj * sc.rk[i] * decay(i, jj) : 0.f;
        }
    }
    if constexpr (!BWD) {
        const int ti = 3 - wave, i = 16 * ti + r;
        for (int tj = 0; tj <= (ti | 1); ++tj) {
            f32x4 m = zero4();
            if (tj <= ti) {
                const f32x4 c = gram(km, tj, qm, ti);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int jj = 16 * tj + 4 * grp + e;
                    m[e] = i >= jj && i < nv ? c[e] * (p.scale * sc.rq[i]) * (sc.rk[jj] * sc.beta[jj]) * decay(i, jj) : 0.f;
                }
            }
            uint8_t *at = rec + R::M + frag_index(ti, tj >> 1) * R::FR + lane * 16 + (tj & 1) * 8;
#pragma unroll
            for (int x = 0; x < X; ++x) {
                const kda::bf16x4 y = kda::to_bf16x4(m);
                *(uint2 *)(at + x * R::MAT) = __builtin_bit_cast(uint2, y);
#pragma unroll
                for (int e = 0; e < 4; ++e) m[e] -= (float)y[e];
            }
        }
    } else {
        // M^T of token tile tj: a lane's four values are consecutive rows i of one column
        const int tj = wave, jj = 16 * tj + r;
        for (int ti = tj & 2; ti < 4; ++ti) {
            f32x4 m = zero4();
            if (ti >= tj) {
                const f32x4 c = gram(qm, ti, km, tj);
                const float sj = p.scale * sc.rk[jj] * sc.beta[jj];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 16 * ti + 4 * grp + e;
                    m[e] = i >= jj && i < nv ? c[e] * sj * sc.rq[i] * decay(i, jj) : 0.f;
                }
            }
            uint8_t *at = rec + R::MT + frag_index_t(tj, ti >> 1) * R::FR + lane * 16 + (ti & 1) * 8;
#pragma unroll
            for (int x = 0; x < X; ++x) {
                const kda::bf16x4 y = kda::to_bf16x4(m);
                *(uint2 *)(at + x * R::MAT) = __builtin_bit_cast(uint2, y);
#pragma unroll
                for (int e = 0; e < 4; ++e) m[e] -= (float)y[e];
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int tj = 0; tj < 4; ++tj)
        if (tj <= wave) block_put(Lm, wave, tj, grp, r, lt[tj]);
    __syncthreads();
    if (wave == 0) {                        // the four diagonal blocks, column r of block grp
        float x[16];
        const float *m = Lm + 16 * grp * P + 16 * grp;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float acc = i == r ? 1.f : 0.f;
#pragma unroll
            for (int jj = 0; jj < i; ++jj) acc -= m[i * P + jj] * x[jj];
            x[i] = acc;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) Xm[(16 * grp + i) * P + 16 * grp + r] = x[i];
    }
    __syncthreads();
    auto a_of = [&](const float *m, int bi, int bj) { return block_a(m, bi, bj, grp, r); };
    auto b_of = [&](const float *m, int bi, int bj) { return block_b(m, bi, bj, grp, r); };
    auto neg = [](f32x4 x) { return f32x4{-x[0], -x[1], -x[2], -x[3]}; };
    if (wave < 2) {                         // X_10 = -X_11 L_10 X_00, X_32 = -X_33 L_32 X_22
        const int lo = 2 * wave, hi = lo + 1;
        const f32x4 t = kda::mm16_f32(a_of(Lm, hi, lo), b_of(Xm, lo, lo), zero4());
        block_put(Xm, hi, lo, grp, r, neg(kda::mm16_f32(a_of(Xm, hi, hi), t, zero4())));
    }
    __syncthreads();
    {                                       // X_ij = -sum_k X_ik (L X)_kj, i = 2, 3, j = 0, 1
        const int i = 2 + (wave >> 1), c = wave & 1;
        auto lx = [&](int row) {
            f32x4 t = kda::mm16_f32(a_of(Lm, row, c), b_of(Xm, c, c), zero4());
            return c == 0 ? kda::mm16_f32(a_of(Lm, row, 1), b_of(Xm, 1, 0), t) : t;
        };
        const f32x4 t2 = lx(2);
        f32x4 x = kda::mm16_f32(a_of(Xm, i, 2), t2, zero4());
        if (i == 3) x = kda::mm16_f32(a_of(Xm, 3, 3), lx(3), x);
        block_put(Xm, i, c, grp, r, neg(x));
    }
    __syncthreads();
    for (int f = wave; f < 6; f += 4) {     // A's fragments
        const int t = f < 2 ? f : 2 + ((f - 2) >> 1), st = f < 2 ? 0 : (f & 1);
        const int i = 16 * t + r;
        f32x4 x[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int c0 = 32 * st + 16 * u + 4 * grp;
            const f32x4 y = *(const f32x4 *)(Xm + i * P + c0);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[u][e] = c0 + e <= i ? y[e] : 0.f;
        }
        const Parts<X> y = split<X>(x[0], x[1]);
        const auto rs = kda::buffer_rsrc(rec, R::BYTES);
#pragma unroll
        for (int k = 0; k < X; ++k)
            kda::bstore16<0>(rs, f * R::FR + lane * 16, R::A + k * R::MAT, y.p[k]);
    }
    if constexpr (BWD) {
        for (int f = wave; f < 6; f += 4) { // A^T's fragments
            const int t = f < 4 ? f >> 1 : f - 2, st = f < 4 ? (f & 1) : 1, jj = 16 * t + r;
            f32x4 x[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 32 * st + 16 * u + 4 * grp + e;
                    x[u][e] = i >= jj ? Xm[i * P + jj] : 0.f;
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

// fp32 x as three bf16 planes: their sum is x to 2^-24 or better
__global__ __launch_bounds__(256) void split_planes_kernel(const float *x, int64_t n4,
                                                           uint2 *planes)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n4) return;
    f32x4 v = ((const f32x4 *)x)[i];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const kda::bf16x4 y = kda::to_bf16x4(v);
        planes[k * n4 + i] = __builtin_bit_cast(uint2, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] -= (float)y[e];
    }
}

hipError_t launch_split_planes(const float *x, int64_t n, uint16_t *planes, hipStream_t st)
{
    const int64_t n4 = n / 4;               // rows are 64 or 128 wide
    if (n4 == 0) return hipSuccess;
    split_planes_kernel<<<dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, st>>>(x, n4,
                                                                                  (uint2 *)planes);
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
