// zero_tail.hip -- the rows behind the last packed sequence set to zero (gdn_zero_tail, include/gdn.h).
//
// The forward and backward kernels leave those rows as they were, and the differentiable calls want zeros there.
// Where they begin lies on the device, so clearing whole tensors ahead would write every output twice; this
// launch writes the tail alone (chunk_gdn, forward and backward, 21412 packed tokens of 32 heads: 2450 -> 2310
// us; a call without a tail takes 6 us, most of it in Python).
#include "gdn.h"
#include "kda_internal.h"

namespace {

constexpr int MAX_TENSORS = 8;

struct Tails {
    const int64_t *cu;                      // the last sequence's end
    int64_t T;
    uint8_t *x[MAX_TENSORS];
    int64_t row_bytes[MAX_TENSORS];
};

// blockIdx.y: the tensor. Rows have an even number of bytes; whole eights between two ends of at most three
// 2-byte stores each.
__global__ __launch_bounds__(256) void zero_tail_kernel(Tails p)
{
    const int64_t from = kda::clamp64(*p.cu, 0, p.T);
    uint8_t *const x = p.x[blockIdx.y];
    const int64_t rb = p.row_bytes[blockIdx.y], b0 = from * rb, b1 = p.T * rb;
    const int64_t up = (b0 + 7) / 8 * 8, lo = up < b1 ? up : b1, down = b1 / 8 * 8, hi = down > lo ? down : lo;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)gridDim.x * 256;
    for (int64_t at = lo + 8 * i; at < hi; at += 8 * n) *(uint2 *)(x + at) = make_uint2(0, 0);
    if (b0 + 2 * i < lo) *(uint16_t *)(x + b0 + 2 * i) = 0;
    if (hi + 2 * i < b1) *(uint16_t *)(x + hi + 2 * i) = 0;
}

}  // namespace

extern "C" kda_status gdn_zero_tail(const int64_t *cu_seqlens, int32_t N, int64_t T, int32_t n, void *const *x,
                                    const int64_t *row_bytes, void *stream)
{
    if (!cu_seqlens || ((uintptr_t)cu_seqlens & 7u) || N < 1 || T < 0 || n < 0 || (n > 0 && (!x || !row_bytes)))
        return KDA_ERR_INVALID_ARG;
    if (n > MAX_TENSORS) return KDA_ERR_UNSUPPORTED;
    Tails p = {};
    p.cu = cu_seqlens + N;
    p.T = T;
    for (int i = 0; i < n; ++i) {
        if (row_bytes[i] < 2 || row_bytes[i] % 2 || (T > 0 && row_bytes[i] > ((int64_t)1 << 62) / T))
            return KDA_ERR_INVALID_ARG;
        if (T > 0 && (!x[i] || ((uintptr_t)x[i] & 7u))) return KDA_ERR_INVALID_ARG;
        p.x[i] = (uint8_t *)x[i];
        p.row_bytes[i] = row_bytes[i];
    }
    if (n == 0 || T == 0) return KDA_OK;
    zero_tail_kernel<<<dim3(256, n), dim3(256), 0, (hipStream_t)stream>>>(p);
    return hipGetLastError() == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}
