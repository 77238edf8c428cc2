// gdn_state.hip -- the forward's pass over a sequence's 64-token chunks (gdn_chain.h).
#include "gdn_segments.h"

namespace gdn {

// C columns of V a workgroup, 16 a wave, two buffers of LDS (one for three planes). 64 columns (a wave on each
// SIMD) have the shortest chunk: 16 heads x 4096 tokens without segments 203 us, against 251 us for 128
// columns in eight waves, 330 us for four waves of 32 columns, 225 us for one buffer and two workgroups a
// compute unit. 128 columns share what is copied to LDS, and their waves hide each other's latencies: bf16
// io with more 64-column workgroups than compute units, all of one length, takes those (whole forward, K = V
// = 128: 5 x 1024 tokens of 32 heads 156 -> 127 us, 8 x 2048 of 32 403 -> 344, 16 x 512 of 32 213 -> 196, K =
// 64: 8 x 1024 of 32 145 -> 121 us). Among packed lengths the longest sequence's chunks count (8 sequences of 3
// .. 8192 tokens, 32 heads, first calls: 471 us with 64 columns, 588 us with 128; repeated 420 us).
template <int K, int V, int C, int IN, int X, bool SEG>
__global__ __launch_bounds__(4 * C) void state_kernel(Params p)
{
    using L = Stage<K, C, IN, Rec<X>, OUT>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[L::BYTES * L::BUFS];
    constexpr int NV = V / C;
    int unit, part;
    if (!unit_of(blockIdx.x, NV, (SEG ? p.seg.slots : p.seq.N) * p.HV, &unit, &part)) return;
    int j = unit % p.HV;
    Segment g;
    const float *init;
    if constexpr (SEG) {
        const int slot = unit / p.HV;
        if (!locate_segment(p.seq, p.seg.chunks, slot, &g)) return;
        init = segment_start<K, V>(p, g, slot, j);
    } else {
        unit = kda::longest_first(p.seq, p.HV, unit);
        j = unit % p.HV;
        g = whole_sequence(p.seq, unit / p.HV);
        init = p.h0 ? p.h0 + (size_t)unit * K * V : nullptr;
    }
    float *const end = p.ht && g.last() ? p.ht + ((size_t)g.s * p.HV + j) * K * V : nullptr;
    forward_chain<K, V, C, IN, X, Rec<X>, OUT>(p, g.s, j, g.c0, g.c1, C * part, init, end, lds);
}

template <int K, int V, int IN, int X>
__global__ __launch_bounds__(256, 2) void ends_kernel(Params p)
{
    using LE = Stage<K, 64, IN, Rec<X>, END>;
    using LP = Stage<K, 64, IN, Rec<X>, PHI>;
    constexpr int A = LE::BYTES * LE::BUFS, B = LP::BYTES * LP::BUFS, NP = V / 64 + K / 64;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[A > B ? A : B];
    int unit, part;
    if (!unit_of(blockIdx.x, NP, p.seg.slots * p.HV, &unit, &part)) return;
    forward_ends<K, V, IN, X, Rec<X>>(p, unit / p.HV, unit % p.HV, part, lds);
}

template <int K, int V, int X>
__global__ __launch_bounds__(256) void join_kernel(Params p)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[Join<K, X>::BYTES];
    int unit, part;
    if (!unit_of(blockIdx.x, V / 16, p.seq.N * p.HV, &unit, &part)) return;
    join_ends<K, V, X, false>(p, p.seg.E, unit / p.HV, unit % p.HV, 16 * part, lds);
}

template <int K, int V, int IN, int X>
hipError_t run(const Params &p, hipStream_t st)
{
    const int64_t units = (int64_t)p.seq.N * p.HV, segs = (int64_t)p.seg.slots * p.HV;
    if (p.seg.chunks == 0) {
        if constexpr (V == 128 && IN == 1) {
            if (!p.seq.cu && 2 * units > kda::current_device_cus()) {
                state_kernel<K, V, 128, IN, X, false><<<dim3(grid_for(units, 1)), dim3(512), 0, st>>>(p);
                return hipGetLastError();
            }
        }
        state_kernel<K, V, 64, IN, X, false><<<dim3(grid_for(units, V / 64)), dim3(256), 0, st>>>(p);
        return hipGetLastError();
    }
    ends_kernel<K, V, IN, X><<<dim3(grid_for(segs, V / 64 + K / 64)), dim3(256), 0, st>>>(p);
    join_kernel<K, V, X><<<dim3(grid_for(units, V / 16)), dim3(256), 0, st>>>(p);
    state_kernel<K, V, 64, IN, X, true><<<dim3(grid_for(segs, V / 64)), dim3(256), 0, st>>>(p);
    return hipGetLastError();
}

template <int K, int V>
hipError_t launch_state(const Params &p, bool f32, hipStream_t st)
{
    return f32 ? run<K, V, 3, 3>(p, st) : run<K, V, 1, 2>(p, st);
}

#define GDN_INST(K, V) template hipError_t launch_state<K, V>(const Params &, bool, hipStream_t);
GDN_INST(64, 64)
GDN_INST(64, 128)
GDN_INST(128, 64)
GDN_INST(128, 128)
#undef GDN_INST

}  // namespace gdn
