// gdn_state.hip -- the forward's pass over a sequence's 64-token chunks (gdn_chain.h).
#include "gdn_chain.h"

namespace gdn {

template <int K, int V, int IN, int X>
__global__ __launch_bounds__(V * 2) void state_kernel(Params p)
{
    using L = Stage<K, V, IN, Rec<X>, true>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[L::BYTES * L::BUFS];
    forward_chain<K, V, IN, X, Rec<X>, true>(p, kda::longest_first(p.seq, p.HV, blockIdx.x), lds, nullptr);
}

template <int K, int V>
hipError_t launch_state(const Params &p, bool f32, hipStream_t st)
{
    const dim3 grid(p.seq.N * p.HV), block(2 * V);
    if (f32)
        state_kernel<K, V, 3, 3><<<grid, block, 0, st>>>(p);
    else
        state_kernel<K, V, 1, 2><<<grid, block, 0, st>>>(p);
    return hipGetLastError();
}

#define GDN_INST(K, V) template hipError_t launch_state<K, V>(const Params &, bool, hipStream_t);
GDN_INST(64, 64)
GDN_INST(64, 128)
GDN_INST(128, 64)
GDN_INST(128, 128)
#undef GDN_INST

}  // namespace gdn
