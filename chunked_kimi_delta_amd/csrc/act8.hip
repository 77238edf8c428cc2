// act8.hip -- activations kept in 8 bits: rows of int8 with one fp32 scale (include/act8.h).
//
// n = round(127 x / m) is decided exactly for bf16 rows: 127 x is exact in fp32 (15 bits), and a
// quotient that is not a tie lies further from one than the correctly rounded division errs.
// fp32 rows divide in 64 bits for the same reason. Both directions stream: a lane takes eight
// values of a row (16 or 32 bytes), a row's maximum is a butterfly over its lanes.
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
// x and m scaled by one power of two, so that m is in [0.5, 1) and 127 x cannot overflow (an x
// that loses bits by it is far below half a step)
__device__ __forceinline__ int quantum(float x, float m, int e, uint16_t) {
    return (int)rintf(127.f * ldexpf(x, -e) / m);
}
__device__ __forceinline__ int quantum(float x, float m, int e, float) {
    return (int)rint(127.0 * (double)ldexpf(x, -e) / (double)m);
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
    u32x2 n = {0, 0};
    if (!bad && !zero) {
        int e;
        const float mm = frexpf(m, &e);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            n[i / 4] |= ((uint32_t)quantum(v[i], mm, e, T()) & 0xffu) << (8 * (i % 4));
    }
    *(u32x2 *)(data + (row * nd + l) * 8) = n;
    if (l == 0) scale[row] = bad ? __uint_as_float(0x7fc00000u) : m / 127.f;
}

__device__ __forceinline__ void store8(uint16_t *p, const float (&x)[8]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i]) |
               (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[2 * i + 1]) << 16;
    ((volatile u32x2 *)p)[0] = u32x2{w[0], w[1]};
    ((volatile u32x2 *)p)[1] = u32x2{w[2], w[3]};
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        ((volatile kda::f32v2 *)p)[i] = kda::f32v2{x[2 * i], x[2 * i + 1]};
}

template <typename T>
__global__ __launch_bounds__(256) void unpack_kernel(const int8_t *data, const float *scale,
                                                     int64_t pieces, int nd, T *x)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= pieces) return;
    const u32x2 n = *(const u32x2 *)(data + i * 8);
    const float s = scale[i / nd];
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)(int8_t)(n[e / 4] >> (8 * (e % 4))) * s;
    store8(x + i * 8, v);
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
    if (rows > ((int64_t)1 << 38) / D) return KDA_ERR_UNSUPPORTED;      // grid limits
    if (rows == 0) return KDA_OK;
    if (!x || !data || !scale || ((uintptr_t)x & 15u) || ((uintptr_t)data & 7u) || ((uintptr_t)scale & 3u))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

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
    const int64_t pieces = rows * (D / 8);
    const dim3 grid((unsigned)((pieces + 255) / 256));
    hipStream_t s = (hipStream_t)stream;
    if (io == KDA_FP32)
        unpack_kernel<<<grid, dim3(256), 0, s>>>(data, scale, pieces, D / 8, (float *)x);
    else
        unpack_kernel<<<grid, dim3(256), 0, s>>>(data, scale, pieces, D / 8, (uint16_t *)x);
    return hipGetLastError() == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
