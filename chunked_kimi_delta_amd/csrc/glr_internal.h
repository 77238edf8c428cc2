// glr_internal.h -- what the kernels of the gated linear recurrence share (include/glr.h).
//
// A token acts on a state as h <- a h + w, a = e^g. Rounding a to 24 bits would make every token of a
// slowly decaying channel err the same way: with g = -1e-5 a state remembers 10^5 tokens, and 2^-25 a
// token adds up to 3e-3 of it. A decay is therefore kept in the form of two numbers (c, s), a = s + c:
// (e^g - 1, 1) where g is in (-1/2, 0], (e^g, 0) elsewhere, and h <- fma(c, h, fma(s, h, w)) holds a's
// distance from 1 to 24 bits as well as a itself.
#pragma once

#include <float.h>

#include <type_traits>

#include "glr.h"
#include "kda_internal.h"

namespace glr {

struct Pre {
    int32_t beta_sigmoid, gate;         // gate: 0 none, 1 softplus, 2 bounded sigmoid
    float lower_bound;
    const float *A_log, *dt_bias;       // [D] (dt_bias may be null)
};

struct Params {
    kda::SeqGeom seq;
    int32_t D, strips;                  // strips: workgroups that share a sequence's channels
    const void *x, *g, *beta;           // beta: null for ones
    int64_t xs, gs, bs;                 // elements from one token to the next
    int64_t xe, ge, be;                 // and from a dense batch's sequence to the next beyond T times as many
    const float *h0;
    void *y;
    float *ht;
    Pre pre;
};

struct BwdParams {
    Params f;                           // f.y: the forward's output
    const void *d_y;
    const float *dht;
    void *dx, *dg, *dbeta;
    float *dh0;
    float *part_A, *part_b;             // [rows][D] sums for dA_log and ddt_bias: of a sequence, or of a tile's slot
};

struct StepParams {
    Params f;
    float *state;
    const int32_t *index;
    int32_t B, T, slots;
};

// ----------------------------------------------------------------------------- scalar functions
//
// On the hardware's base-2 exponential and its reciprocal (1 ulp each). fp32 io adds what the product
// with log2 e rounds away and a Newton step, since an fp32 output would show them; bf16 io does not.

template <typename T>
__device__ __forceinline__ float exp_(float x) {
    const float t = x * kda::LOG2E, r = __builtin_amdgcn_exp2f(t);
    if constexpr (sizeof(T) == 2) return r;
    // x log2 e = t + lo. Where r is infinite (t >= 128) or x is, lo must not make a NaN of it: t in (-160, 128) only
    const float lo = fmaf(x, 1.925963033500931e-8f, fmaf(x, kda::LOG2E, -t));
    return fabsf(t + 16.f) < 144.f ? fmaf(r, lo * 0.6931471805599453f, r) : r;
}
template <typename T>
__device__ __forceinline__ float inverse(float x) {     // of x in [1, 2]
    const float r = __builtin_amdgcn_rcpf(x);
    if constexpr (sizeof(T) == 2) return r;
    return fmaf(fmaf(-x, r, 1.f), r, r);
}
// log(1 + e) of e in [0, 1]: e p(e), p fitted there (bf16 io 2^-22 of it off, fp32 io 2^-24)
template <typename T>
__device__ __forceinline__ float log1p_(float e) {
    float p;
    if constexpr (sizeof(T) == 2) {
        p = -0.00857467577f;
        p = fmaf(p, e, 0.0442141928f);
        p = fmaf(p, e, -0.107853681f);
        p = fmaf(p, e, 0.177570239f);
        p = fmaf(p, e, -0.244996116f);
        p = fmaf(p, e, 0.332761765f);
        p = fmaf(p, e, -0.499974489f);
        p = fmaf(p, e, 0.999999821f);
    } else {
        p = -0.00325637846f;
        p = fmaf(p, e, 0.0199071616f);
        p = fmaf(p, e, -0.0570642017f);
        p = fmaf(p, e, 0.106142648f);
        p = fmaf(p, e, -0.153118625f);
        p = fmaf(p, e, 0.196781173f);
        p = fmaf(p, e, -0.249545589f);
        p = fmaf(p, e, 0.333300054f);
        p = fmaf(p, e, -0.499999046f);
        p = fmaf(p, e, 1.f);
    }
    return e * p;
}

// sigmoid and its derivative from e^-|x|, each to a few roundings of itself
struct Sigmoid {
    float s, ds;
};
template <typename T>
__device__ __forceinline__ Sigmoid sigmoid(float x) {
    const float e = exp_<T>(-fabsf(x)), r = inverse<T>(1.f + e), o = e * r;
    return Sigmoid{x < 0.f ? o : r, o * r};
}

// the sigmoid alone
template <typename T>
__device__ __forceinline__ float logistic(float x) {
    if constexpr (sizeof(T) == 2) return __builtin_amdgcn_rcpf(1.f + exp_<T>(-x));
    return sigmoid<T>(x).s;
}

// e^g - 1 for g in [-1/2, 0]: g + g^2 q(g), q fitted there (2^-26 of the whole off)
__device__ __forceinline__ float expm1_slow(float g) {
    float q = 0.0011646067f;
    q = fmaf(q, g, 0.008238542f);
    q = fmaf(q, g, 0.04165003f);
    q = fmaf(q, g, 0.16666564f);
    q = fmaf(q, g, 0.5f);
    return fmaf(g * g, q, g);
}

// e^g as (c, s)
template <typename T>
__device__ __forceinline__ void decay(float g, float &c, float &s) {
    const bool slow = fabsf(g + 0.25f) <= 0.25f;
    float d = expm1_slow(g), a = exp_<T>(g);
    asm("" : "+v"(d), "+v"(a));         // both, and no branch around either
    c = slow ? d : a;
    s = slow ? 1.f : 0.f;
}

// A channel's gate. active() is the log decay of a raw input; back() takes the gradient dg of the active
// decay `act` to that of the raw input and adds to the gradients of A_log and dt_bias. The kind is a type, so
// that a lane's tokens go through one branch together. An infinite input (a state cleared or kept) has no part in
// A_log's gradient, nor has a far one: there dg or du is zero, and the other factor is taken as finite.
enum Kind { NONE, SOFTPLUS, BOUNDED };

struct Gate {
    float ea, bias, lb;

    template <typename T, Kind N>
    __device__ __forceinline__ float active(float g) const {
        if (N == NONE) return g;
        const float u = g + bias;
        if (N == SOFTPLUS) return -ea * (fmaxf(u, 0.f) + log1p_<T>(exp_<T>(-fabsf(u))));
        return lb * logistic<T>(ea * u);
    }
    template <typename T, Kind N>
    __device__ __forceinline__ float back(float g, float act, float dg, float &dA, float &db) const {
        if (N == NONE) return dg;
        const float u = g + bias;
        const float du = N == SOFTPLUS ? -ea * logistic<T>(u) * dg : ea * lb * sigmoid<T>(ea * u).ds * dg;
        dA += N == SOFTPLUS ? fmaxf(act, -FLT_MAX) * dg : du * __builtin_amdgcn_fmed3f(u, -FLT_MAX, FLT_MAX);
        db += du;
        return du;
    }
};
template <class Fn>
__device__ __forceinline__ void by_kind(int kind, Fn fn) {
    if (kind == 0) fn(std::integral_constant<Kind, NONE>());
    else if (kind == 1) fn(std::integral_constant<Kind, SOFTPLUS>());
    else fn(std::integral_constant<Kind, BOUNDED>());
}

__device__ __forceinline__ Gate gate_of(const Pre &pre, int d) {
    Gate g = {1.f, 0.f, pre.lower_bound};
    if (pre.gate) {
        g.ea = expf(pre.A_log[d]);
        if (pre.dt_bias) g.bias = pre.dt_bias[d];
    }
    return g;
}

// ----------------------------------------------------------------------------- a lane's channels
//
// VEC neighbouring channels of one token, as they are stored; loads past a resource's range give zeros,
// stores past it are dropped.

// No resource reaches PAST (2^29 bytes at most: 512 rows of 2^18 fp32 values), nor do PAST less or more as much.
constexpr uint32_t PAST = 0xc0000000u;

template <typename T, int VEC> struct Raw;
template <int VEC> struct Raw<uint16_t, VEC> { uint32_t v; };
template <int VEC> struct Raw<float, VEC> { float v[VEC]; };

__device__ __forceinline__ void load(Raw<uint16_t, 1> &r, __amdgpu_buffer_rsrc_t b, uint32_t off) {
    r.v = (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, off, 0, 0);
}
__device__ __forceinline__ void load(Raw<uint16_t, 2> &r, __amdgpu_buffer_rsrc_t b, uint32_t off) {
    r.v = __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0);
}
__device__ __forceinline__ void load(Raw<float, 1> &r, __amdgpu_buffer_rsrc_t b, uint32_t off) {
    r.v[0] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0));
}
__device__ __forceinline__ void load(Raw<float, 2> &r, __amdgpu_buffer_rsrc_t b, uint32_t off) {
    const kda::f32v2 v = __builtin_bit_cast(kda::f32v2, __builtin_amdgcn_raw_buffer_load_b64(b, off, 0, 0));
    r.v[0] = v[0];
    r.v[1] = v[1];
}

template <int VEC>
__device__ __forceinline__ float value(const Raw<uint16_t, VEC> &r, int i) { return i ? kda::bf16hi(r.v) : kda::bf16lo(r.v); }
template <int VEC>
__device__ __forceinline__ float value(const Raw<float, VEC> &r, int i) { return r.v[i]; }

__device__ __forceinline__ uint32_t bf16_bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ uint32_t bf16_bits(float x, float y) {
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x, (__bf16)y});
}
template <typename T, int VEC>
__device__ __forceinline__ void store(const float (&v)[VEC], __amdgpu_buffer_rsrc_t b, uint32_t off) {
    if constexpr (sizeof(T) == 2 && VEC == 1)
        __builtin_amdgcn_raw_buffer_store_b16((uint16_t)bf16_bits(v[0]), b, off, 0, 0);
    else if constexpr (sizeof(T) == 2)
        __builtin_amdgcn_raw_buffer_store_b32(bf16_bits(v[0], v[1]), b, off, 0, 0);
    else if constexpr (VEC == 1)
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v[0]), b, off, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(kda::u32x2, kda::f32v2{v[0], v[1]}), b, off, 0, 0);
}

// A lane's log decays of N tokens, and the sums, least and largest of them. live: tokens that the sequence has
// from the lane's first on (a raw gate input of zero is no log decay of zero).
template <typename T, int N, int VEC>
__device__ __forceinline__ void log_decays(const Raw<T, VEC> (&raw)[N], const Gate (&gate)[VEC], int kind, int live,
                                           float (&g)[N][VEC], float (&G)[VEC], float &least, float &most) {
    by_kind(kind, [&](auto n) {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) g[k][v] = gate[v].template active<T, decltype(n)::value>(value(raw[k], v));
    });
    if (kind != 0 && live < N) {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) g[k][v] = k < live ? g[k][v] : 0.f;
    }
    least = most = g[0][0];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        G[v] = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            G[v] += g[k][v];
            least = fminf(least, g[k][v]);
            most = fmaxf(most, g[k][v]);
        }
    }
}
// x beta
template <typename T, int N, int VEC>
__device__ __forceinline__ void gated_inputs(const Raw<T, VEC> (&x)[N], const Raw<T, VEC> (&beta)[N], int is_logit,
                                             float (&w)[N][VEC]) {
    if (is_logit) {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) w[k][v] = value(x[k], v) * logistic<T>(value(beta[k], v));
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v) w[k][v] = value(x[k], v) * value(beta[k], v);
    }
}

// Host-side launchers (defined next to their kernels). vec: channels a lane; lanes: lanes a token
// (Params.strips = ceil(D / (vec lanes))).
struct Shape {
    bool f32, tiles;
    int vec, lanes;
};
hipError_t launch_fwd(const Params &p, Shape s, hipStream_t st);
hipError_t launch_bwd(const BwdParams &p, Shape s, hipStream_t st);
hipError_t launch_params(const BwdParams &p, int64_t rows, float *dA_log, float *ddt_bias, hipStream_t st);
// the same in tiles (64 lanes a token): workspace bytes, and for the backward rows of its partial sums
int64_t tiles_bytes(const Params &p, Shape s);
hipError_t launch_fwd_tiles(const Params &p, Shape s, void *ws, hipStream_t st);
int64_t tiles_back_bytes(const Params &p, Shape s);
int64_t tiles_back_rows(const Params &p);
hipError_t launch_bwd_tiles(const BwdParams &p, Shape s, void *ws, hipStream_t st);
hipError_t launch_step(const StepParams &p, bool f32, int vec, hipStream_t st);

constexpr int W = 8, K = 8;             // waves a workgroup and tokens a lane and step of the strips' kernels

}  // namespace glr
