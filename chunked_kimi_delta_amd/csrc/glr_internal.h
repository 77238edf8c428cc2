// glr_internal.h -- what the kernels of the gated linear recurrence share (include/glr.h).
//
// A token acts on a state as h <- a h + w, a = e^g. Rounding a to 24 bits would make every token of a
// slowly decaying channel err the same way: with g = -1e-5 a state remembers 10^5 tokens, and 2^-25 a
// token adds up to 3e-3 of it. A decay is therefore kept in the form of two numbers (c, s), a = s + c:
// (e^g - 1, 1) where g is in (-1/2, 0], (e^g, 0) elsewhere, and h <- fma(c, h, fma(s, h, w)) holds a's
// distance from 1 to 24 bits as well as a itself.
#pragma once

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
    float *part_A, *part_b;             // [N][D] a sequence's sums for dA_log and ddt_bias
};

struct StepParams {
    Params f;
    float *state;
    const int32_t *index;
    int32_t B, T, slots;
};

// ----------------------------------------------------------------------------- scalar functions
//
// bf16 io takes the hardware's base-2 functions (1 ulp each), fp32 io the library's: an fp32 output
// shows what a product with log2 e rounds away from a large argument, a bf16 one does not.

template <typename T> __device__ __forceinline__ float exp_(float x);
template <> __device__ __forceinline__ float exp_<uint16_t>(float x) { return __builtin_amdgcn_exp2f(x * kda::LOG2E); }
template <> __device__ __forceinline__ float exp_<float>(float x) { return expf(x); }

template <typename T> __device__ __forceinline__ float inverse(float x);
template <> __device__ __forceinline__ float inverse<uint16_t>(float x) { return __builtin_amdgcn_rcpf(x); }
template <> __device__ __forceinline__ float inverse<float>(float x) { return 1.f / x; }

// sigmoid and its derivative from e^-|x|, each to a few roundings of itself
struct Sigmoid {
    float s, ds;
};
template <typename T>
__device__ __forceinline__ Sigmoid sigmoid(float x) {
    const float e = exp_<T>(-fabsf(x)), r = inverse<T>(1.f + e), o = e * r;
    return Sigmoid{x < 0.f ? o : r, o * r};
}

// e^g as (c, s). On (-1/2, 0] e^g - 1 = g + g^2 q(g), with a q of degree 4 fitted there (2^-26 of
// e^g - 1 off).
template <typename T>
__device__ __forceinline__ void decay(float g, float &c, float &s) {
    float q = 0.0011646067f;
    q = fmaf(q, g, 0.008238542f);
    q = fmaf(q, g, 0.04165003f);
    q = fmaf(q, g, 0.16666564f);
    q = fmaf(q, g, 0.5f);
    const bool slow = g > -0.5f && g <= 0.f;
    c = slow ? fmaf(g * g, q, g) : exp_<T>(g);
    s = slow ? 1.f : 0.f;
}

// A channel's gate. active() is the log decay of a raw input; back() takes the gradient of the active
// decay to that of the raw input and adds to the gradients of A_log and dt_bias.
template <typename T>
struct Gate {
    int kind;
    float ea, bias, lb;

    // log(1 + e^u) from e = e^-|u|: log1p(e) = log w + (e - (w - 1)) / w, w = 1 + e rounded
    __device__ __forceinline__ float softplus(float u) const {
        if constexpr (sizeof(T) == 4) {
            return fmaxf(u, 0.f) + log1pf(expf(-fabsf(u)));
        } else {
            const float e = exp_<T>(-fabsf(u)), w = 1.f + e;
            return fmaxf(u, 0.f) + fmaf(__builtin_amdgcn_logf(w), 0.6931471805599453f, (e - (w - 1.f)) * inverse<T>(w));
        }
    }
    __device__ __forceinline__ float active(float g) const {
        if (kind == 0) return g;
        const float u = g + bias;
        return kind == 1 ? -ea * softplus(u) : lb * sigmoid<T>(ea * u).s;
    }
    __device__ __forceinline__ float back(float g, float dg, float &dA, float &db) const {
        const float u = g + bias;
        if (kind == 1) {
            const float du = -ea * sigmoid<T>(u).s * dg;
            dA -= ea * softplus(u) * dg;
            db += du;
            return du;
        }
        const float du = ea * lb * sigmoid<T>(ea * u).ds * dg;
        dA += du * u;
        db += du;
        return du;
    }
};

template <typename T>
__device__ __forceinline__ Gate<T> gate_of(const Pre &pre, int d) {
    Gate<T> g = {pre.gate, 1.f, 0.f, pre.lower_bound};
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
template <typename T, int VEC>
__device__ __forceinline__ void store(const float (&v)[VEC], __amdgpu_buffer_rsrc_t b, uint32_t off) {
    if constexpr (sizeof(T) == 2 && VEC == 1)
        __builtin_amdgcn_raw_buffer_store_b16((uint16_t)bf16_bits(v[0]), b, off, 0, 0);
    else if constexpr (sizeof(T) == 2)
        __builtin_amdgcn_raw_buffer_store_b32(bf16_bits(v[0]) | bf16_bits(v[1]) << 16, b, off, 0, 0);
    else if constexpr (VEC == 1)
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v[0]), b, off, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(kda::u32x2, kda::f32v2{v[0], v[1]}), b, off, 0, 0);
}

// Host-side launchers (defined next to their kernels). vec: channels a lane; lanes: lanes a token
// (Params.strips = ceil(D / (vec lanes))).
struct Shape {
    bool f32;
    int vec, lanes;
};
hipError_t launch_fwd(const Params &p, Shape s, hipStream_t st);
hipError_t launch_bwd(const BwdParams &p, Shape s, hipStream_t st);
hipError_t launch_params(const BwdParams &p, float *dA_log, float *ddt_bias, hipStream_t st);
hipError_t launch_step(const StepParams &p, bool f32, int vec, hipStream_t st);

constexpr int W = 8, K = 8;             // waves a workgroup, tokens a lane and step

}  // namespace glr
