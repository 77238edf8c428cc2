// act8.hip -- activations kept in 8 bits: rows of int8 with one fp32 scale (include/act8.h).
//
// Both directions stream, so what counts is the bytes and few instructions a value. Packing rounds
// 127 x / m. A product with an approximate 127 / m decides that except within 2^-16 of a tie; what is left
// of 127 x tells which: d = 127 x - n m is exact for bf16 rows (15 bits each), and n stands where
// |2 d| < m. Where a wave holds a value that may not, it divides (correctly rounded, which decides every
// case of bf16 exactly); fp32 rows divide in 64 bits. A lane takes eight values of a row, and a row's
// maximum is a butterfly over its lanes. Unpacking writes eight bytes a lane, whole lines a store. 4096 x 48 rows
// of 128 bf16: packing 18.3 us (4.2 TB/s, its vector instructions; first calls 19.4, with two rows a lane 21, with
// four 24 us: loads in flight are not what it lacks), unpacking 14.4 us (5.3 TB/s, what a copy reaches). fp32 rows: 23.5
// and 20.3 us (5.4 and 6.2 TB/s, part of it from the last-level cache).
#include "act8.h"
#include "kda_internal.h"

namespace {

using kda::u32x2;
using kda::u32x4;

template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
#pragma unroll
    for (int m = LPR / 2; m >= 1; m >>= 1) {
        const uint32_t y = (uint32_t)__shfl_xor((int)x, m);
        x = x > y ? x : y;
    }
    return x;
}

__device__ __forceinline__ void load8(const uint16_t *p, float (&x)[8]) {
    const u32x4 v = *(const u32x4 *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = kda::bf16lo(v[i]);
        x[2 * i + 1] = kda::bf16hi(v[i]);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const kda::f32x4 a = *(const kda::f32x4 *)p, b = *(const kda::f32x4 *)(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = a[i];
        x[4 + i] = b[i];
    }
}
// round(127 x / m) of eight values, m their row's largest magnitude: whole numbers as floats. x and m are
// scaled by one power of two, so that m is in [0.5, 1) and 127 x cannot overflow (an x that loses bits by
// it is far below half a step).
__device__ __forceinline__ void quanta(const float (&v)[8], float m, float (&n)[8], uint16_t) {
    int e;
    const float mm = frexpf(m, &e), s = 127.f * __builtin_amdgcn_rcpf(mm);
    bool near = false;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = ldexpf(v[i], -e);
        n[i] = __builtin_rintf(x[i] * s);
        const float d = fmaf(-n[i], mm, 127.f * x[i]);
        near |= fabsf(d + d) >= mm;
    }
    if (__builtin_amdgcn_ballot_w64(near)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = __builtin_rintf(127.f * x[i] / mm);
    }
}
__device__ __forceinline__ void quanta(const float (&v)[8], float m, float (&n)[8], float) {
    int e;
    const double mm = (double)frexpf(m, &e);
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = (float)rint(127.0 * (double)ldexpf(v[i], -e) / mm);
}
// four whole numbers in [-127, 127] as bytes: behind 1.5 x 2^23 a float's low byte is the number
__device__ __forceinline__ uint32_t bytes4(float a, float b, float c, float d) {
    auto bits = [](float x) { return __float_as_uint(x + 12582912.f); };
    const uint32_t lo = __builtin_amdgcn_perm(bits(b), bits(a), 0x0c0c0400u), hi = __builtin_amdgcn_perm(bits(d), bits(c), 0x0c0c0400u);
    return lo | hi << 16;
}

// Rows of D = 8 ND values, LPR >= ND lanes a row (a power of two).
template <int LPR, typename T>
__global__ __launch_bounds__(256) void pack_kernel(const T *x, int64_t rows, int nd, int8_t *data,
                                                   float *scale)
{
    const int64_t row = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int l = threadIdx.x % LPR;
    const bool on = row < rows && l < nd;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (on) load8(x + (row * nd + l) * 8, v);
    uint32_t most = 0;                      // bits of the largest magnitude; NaN is above inf
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
        most = most > u ? most : u;
    }
    most = row_max<LPR>(most);
    if (!on) return;
    const bool bad = most >= 0x7f800000u, zero = most == 0;
    const float m = __uint_as_float(most);
    float q[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (!bad && !zero) quanta(v, m, q, T());
    const u32x2 n = {bytes4(q[0], q[1], q[2], q[3]), bytes4(q[4], q[5], q[6], q[7])};
    *(u32x2 *)(data + (row * nd + l) * 8) = n;
    if (l == 0) scale[row] = bad ? __uint_as_float(0x7fc00000u) : m / 127.f;
}

// One tensor of an unpacking launch: rows of 4 << shift values (shift >= 0), or 4 nq values.
struct Unpack {
    const int8_t *data;
    const float *scale;
    void *x;
    int64_t quads;                          // groups of four values
    int32_t nq, shift;
};
struct Unpacks {
    Unpack t[3];
};

// Four values a lane: four bytes in, eight (sixteen: two stores of eight) out.
template <typename T>
__device__ __forceinline__ void unpack4(const Unpack &u, int64_t i) {
    const uint32_t n = ((const uint32_t *)u.data)[i];
    const float s = u.scale[u.shift >= 0 ? i >> u.shift : i / u.nq];
    const kda::f32x4 v = kda::f32x4{(float)(int8_t)n, (float)(int8_t)(n >> 8), (float)(int8_t)(n >> 16),
                                    (float)(int8_t)(n >> 24)} * s;
    if constexpr (sizeof(T) == 2)
        ((uint2 *)u.x)[i] = __builtin_bit_cast(uint2, kda::to_bf16x4(v));
    else
        kda::bstore16<0>(kda::buffer_rsrc((kda::f32x4 *)u.x + (i - threadIdx.x), 4096), threadIdx.x * 16, 0, v);
}

// Tensors one behind the other, each from a whole block on.
template <typename T>
__global__ __launch_bounds__(256) void unpack_kernel(Unpacks p)
{
    int64_t block = blockIdx.x;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int64_t blocks = (p.t[k].quads + 255) / 256;
        if (block < blocks) {
            const int64_t i = block * 256 + threadIdx.x;
            if (i < p.t[k].quads) unpack4<T>(p.t[k], i);
            return;
        }
        block -= blocks;
    }
}

Unpack unpack_of(const int8_t *data, const float *scale, int64_t rows, int32_t D, void *x)
{
    const int nq = D / 4;
    return Unpack{data, scale, x, rows * nq, nq, (nq & (nq - 1)) == 0 ? __builtin_ctz(nq) : -1};
}

hipError_t launch_unpack(const Unpacks &p, bool f32, hipStream_t st)
{
    int64_t blocks = 0;
    for (const Unpack &u : p.t) blocks += (u.quads + 255) / 256;
    if (blocks == 0) return hipSuccess;
    if (f32)
        unpack_kernel<float><<<dim3((unsigned)blocks), dim3(256), 0, st>>>(p);
    else
        unpack_kernel<uint16_t><<<dim3((unsigned)blocks), dim3(256), 0, st>>>(p);
    return hipGetLastError();
}

template <int LPR>
void launch_pack(const void *x, bool f32, int64_t rows, int nd, int8_t *data, float *scale,
                 hipStream_t st)
{
    const dim3 grid((unsigned)((rows + 256 / LPR - 1) / (256 / LPR)));
    if (f32)
        pack_kernel<LPR, float><<<grid, dim3(256), 0, st>>>((const float *)x, rows, nd, data, scale);
    else
        pack_kernel<LPR, uint16_t><<<grid, dim3(256), 0, st>>>((const uint16_t *)x, rows, nd, data, scale);
}

kda_status check(const void *x, int32_t io, int64_t rows, int32_t D, const void *data,
                 const void *scale)
{
    if (rows < 0 || D < 8 || D % 8) return KDA_ERR_INVALID_ARG;
    if (D > 512 || (io != KDA_BF16 && io != KDA_FP32)) return KDA_ERR_UNSUPPORTED;
    // less than 2^32 lanes: below D / 4 a row, but four for D = 8, in whole blocks of up to 64 rows
    if (rows >= ((int64_t)1 << 33) / D || rows > ((int64_t)1 << 30) - 64) return KDA_ERR_UNSUPPORTED;
    if (rows == 0) return KDA_OK;
    if (!x || !data || !scale || ((uintptr_t)x & 15u) || ((uintptr_t)data & 7u) || ((uintptr_t)scale & 3u))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

namespace gdn {

hipError_t launch_unpack3(const int8_t *const data[3], const float *const scale[3], const int64_t rows[3],
                          const int32_t D[3], void *const x[3], bool f32, hipStream_t st)
{
    Unpacks p;
    for (int i = 0; i < 3; ++i) p.t[i] = unpack_of(data[i], scale[i], rows[i], D[i], x[i]);
    return launch_unpack(p, f32, st);
}

}  // namespace gdn

extern "C" {

kda_status act8_pack(const void *x, int32_t io, int64_t rows, int32_t D, int8_t *data,
                     float *scale, void *stream)
{
    const kda_status st = check(x, io, rows, D, data, scale);
    if (st != KDA_OK || rows == 0) return st;
    const int nd = D / 8;
    const bool f32 = io == KDA_FP32;
    hipStream_t s = (hipStream_t)stream;
    if (nd <= 4) launch_pack<4>(x, f32, rows, nd, data, scale, s);
    else if (nd <= 8) launch_pack<8>(x, f32, rows, nd, data, scale, s);
    else if (nd <= 16) launch_pack<16>(x, f32, rows, nd, data, scale, s);
    else if (nd <= 32) launch_pack<32>(x, f32, rows, nd, data, scale, s);
    else launch_pack<64>(x, f32, rows, nd, data, scale, s);
    return hipGetLastError() == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status act8_unpack(const int8_t *data, const float *scale, int32_t io, int64_t rows,
                       int32_t D, void *x, void *stream)
{
    const kda_status st = check(x, io, rows, D, data, scale);
    if (st != KDA_OK || rows == 0) return st;
    Unpacks p = {};
    p.t[0] = unpack_of(data, scale, rows, D, x);
    return launch_unpack(p, io == KDA_FP32, (hipStream_t)stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
