// gdn_state.hip -- the forward's pass over a sequence's 64-token chunks (gdn_chain.h).
#include "gdn_chain.h"

namespace gdn {

// Columns of a workgroup: all of V, or 64 of 128 where the batch leaves compute units idle
// (two workgroups a unit, each with half the work per chunk).
template <int K, int V, int C, int IN, int X>
__global__ __launch_bounds__(C * 4) void state_kernel(Params p)
{
    using L = Stage<K, C, IN, Rec<X>, OUT>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[L::BYTES * L::BUFS];
    const int unit = kda::longest_first(p.seq, p.HV, blockIdx.x / (V / C)), part = blockIdx.x % (V / C);
    const int s = unit / p.HV, j = unit % p.HV;
    const int64_t bos = kda::seq_bos(p.seq, s), eos = kda::seq_eos(p.seq, s, bos);
    const size_t at = ((size_t)s * p.HV + j) * K * V;
    forward_chain<K, V, C, IN, X, Rec<X>, OUT>(p, s, j, 0, (int)((eos - bos + CT - 1) / CT), part * C,
                                               p.h0 ? p.h0 + at : nullptr, p.ht ? p.ht + at : nullptr, lds);
}

template <int K, int V>
hipError_t launch_state(const Params &p, bool f32, hipStream_t st)
{
    const unsigned units = p.seq.N * p.HV;
    const bool halves = V == 128 && 2 * (int64_t)units <= kda::current_device_cus();
    if (f32)
        state_kernel<K, V, 64, 3, 3><<<dim3(units * (V / 64)), dim3(256), 0, st>>>(p);
    else if (halves || V == 64)
        state_kernel<K, V, 64, 1, 2><<<dim3(units * (V / 64)), dim3(256), 0, st>>>(p);
    else
        state_kernel<K, V, V, 1, 2><<<dim3(units), dim3(4 * V), 0, st>>>(p);
    return hipGetLastError();
}

#define GDN_INST(K, V) template hipError_t launch_state<K, V>(const Params &, bool, hipStream_t);
GDN_INST(64, 64)
GDN_INST(64, 128)
GDN_INST(128, 64)
GDN_INST(128, 128)
#undef GDN_INST

}  // namespace gdn
