// gdn_state.hip -- the forward's pass over a sequence's 64-token chunks (gdn_chain.h).
#include "gdn_chain.h"

namespace gdn {

// C columns of V a workgroup, CTW 16-column tiles a wave.
template <int K, int V, int C, int CTW, int IN, int X>
__global__ __launch_bounds__(C * 4 / CTW) void state_kernel(Params p)
{
    using L = Stage<K, C, IN, Rec<X>, OUT>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[L::BYTES * L::BUFS];
    const int unit = kda::longest_first(p.seq, p.HV, blockIdx.x / (V / C)), part = blockIdx.x % (V / C);
    const int s = unit / p.HV, j = unit % p.HV;
    const int64_t bos = kda::seq_bos(p.seq, s), eos = kda::seq_eos(p.seq, s, bos);
    const size_t at = ((size_t)s * p.HV + j) * K * V;
    forward_chain<K, V, C, CTW, IN, X, Rec<X>, OUT>(p, s, j, 0, (int)((eos - bos + CT - 1) / CT), part * C,
                                                    p.h0 ? p.h0 + at : nullptr, p.ht ? p.ht + at : nullptr, lds);
}

template <int K, int V, int C, int CTW, int IN, int X>
void run(const Params &p, hipStream_t st)
{
    state_kernel<K, V, C, CTW, IN, X><<<dim3(p.seq.N * p.HV * (V / C)), dim3(C * 4 / CTW), 0, st>>>(p);
}

template <int K, int V>
hipError_t launch_state(const Params &p, bool f32, hipStream_t st)
{
    if (f32)
        run<K, V, 64, 1, 3, 3>(p, st);
    else
        run<K, V, 64, 1, 1, 2>(p, st);
    return hipGetLastError();
}

#define GDN_INST(K, V) template hipError_t launch_state<K, V>(const Params &, bool, hipStream_t);
GDN_INST(64, 64)
GDN_INST(64, 128)
GDN_INST(128, 64)
GDN_INST(128, 128)
#undef GDN_INST

}  // namespace gdn
