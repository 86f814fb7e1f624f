// Arguments and the token's mathematics of the gated linear recurrence
// (lru.hip, lru_bwd.hip): for each channel
//     log a_t = -rate sigma(r_t), s_t = sqrt(1 - a_t^2)   with a rate,
//     a_t = sigma(r_t),           s_t = 1 - a_t           without,
//     h_t = a_t h_{t-1} + s_t sigma(i_t) x_t,   y_t = h_t.
// a and o = 1 - a are both kept to their relative accuracy: s comes from o
// (1 - a^2 = o (2 - o)), which a difference from a near 1 would have lost.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "vec.hpp"

namespace ttt {

struct LruArgs {
    int B, L, D, io;
    const void *x, *r, *i;  // [B,L,D]; i may be null
    int64_t xb, xt, rb, rt, ib, it;
    const float *rate;   // [D] or null
    const float *state;  // [B,D] or null
    const int *lens;     // [B] or null
    void *y;
    int64_t yb, yt;
    float *state_out;  // [B,D] or null
    float *ws;
};

struct LruBwdArgs {
    LruArgs f;  // forward arguments (y, state_out unused)
    const void *dy;
    int64_t dyb, dyt;
    const float *dstate_out;  // [B,D] or null
    void *dx, *dr, *di;
    int64_t dxb, dxt, drb, drt, dib, dit;
    float *drate, *dstate;
};

hipError_t launch_lru_forward(const LruArgs &a, hipStream_t stream);
hipError_t launch_lru_step(const LruArgs &a, hipStream_t stream);  // state_out read and written
hipError_t launch_lru_backward(const LruBwdArgs &a, hipStream_t stream);
int64_t lru_forward_floats(int B, int L, int D);   // workspace
int64_t lru_backward_floats(int B, int L, int D);

namespace lru {

constexpr int NT = 256;     // threads of a workgroup
constexpr int CH = 128;     // channels of its tile

__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// e^z and o = 1 - e^z for z <= 0. Where e^z is near 1, o comes from the series
// (the next term is below 2^-25 of it at -0.1, where 1 - e^z is off by 2^-20.6
// at most) and e^z from o.
__device__ __forceinline__ float decay(float z, float *o) {
    float p = fmaf(z, 1.0f / 5, 1.0f);
    p = fmaf(z * 0.25f, p, 1.0f);
    p = fmaf(z * (1.0f / 3), p, 1.0f);
    p = fmaf(z * 0.5f, p, 1.0f);
    const float e = fast_exp(z);
    *o = z > -0.1f ? -z * p : 1.0f - e;
    return z > -0.1f ? 1.0f - *o : e;
}

// sigma(v) and 1 - sigma(v)
__device__ __forceinline__ float sigmoid2(float v, float *other) {
    const float t = fast_exp(-fabsf(v)), d = __builtin_amdgcn_rcpf(1.0f + t), q = t * d;
    *other = v >= 0.f ? q : d;
    return v >= 0.f ? d : q;
}
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + fast_exp(-v)); }

// What a token's gate comes to.
struct Gate {
    float a, o;  // the decay, 1 - a
    float s;     // the input's scale
    float g, ng; // with a rate: sigma(r), 1 - sigma(r)
};

// Rates are >= 0. A closed gate (r = -infinity) gives a = 1, o = s = 0.
template <bool RATE> __device__ __forceinline__ Gate gate(float r, float rate) {
    Gate k;
    if constexpr (RATE) {
        k.g = sigmoid2(r, &k.ng);
        k.a = decay(-rate * k.g, &k.o);
        k.s = __builtin_amdgcn_sqrtf(k.o * (2.0f - k.o));
    } else {
        k.a = sigmoid2(r, &k.o);
        k.s = k.o;
        k.g = k.ng = 0.f;
    }
    return k;
}

}  // namespace lru
}  // namespace ttt
