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
// tokens of a prompt's tile where a thread takes V channels
int lru_forward_tokens(int B, int L, int D, int V, bool gated);

namespace lru {

constexpr int NT = 256;     // threads of a workgroup
constexpr int CH = 128;     // channels of its tile

constexpr float LOG2E = 1.44269504f;

__device__ __forceinline__ int live_tokens(const int *lens, int b, int L) {
    return lens ? max(0, min(lens[b], L)) : L;
}
// A tile with all of its tokens (of a sequence of n) and channels, as nearly all are: its loops
// ask for no token's or channel's place, whose branches cost copies of what is held across them.
__device__ __forceinline__ bool whole(int tile, int tokens, int n, int c0, int D) {
    return (tile + 1) * tokens <= n && c0 + CH <= D;
}

// A value to a thread, for any number of them: a grid's threads are counted in 32 bits along each
// of its dimensions, so the workgroups go on in the second after MOST.
constexpr int MOST = 1 << 22;
inline dim3 values_grid(int64_t n) {
    const int64_t g = (n + NT - 1) / NT;
    return dim3(static_cast<unsigned>(g < MOST ? g : MOST), static_cast<unsigned>((g + MOST - 1) / MOST));
}
__device__ __forceinline__ int64_t value_at() {
    return (static_cast<int64_t>(blockIdx.y) * MOST + blockIdx.x) * NT + threadIdx.x;
}

inline bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * LOG2E); }
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + fast_exp(-v)); }
// sigma(v) and 1 - sigma(v) = e^-v sigma(v), which is 1 where e^-v is out of the reciprocal's range
__device__ __forceinline__ float sigmoid2(float v, float *other) {
    const float t = fast_exp(-v), d = __builtin_amdgcn_rcpf(1.0f + t);
    *other = t > 1e37f ? 1.0f : t * d;
    return d;
}

// 2^z and o = 1 - 2^z for z <= 0. Where 2^z is near 1, o comes from the series of
// 1 - e^(z ln 2) (the next term is below 2^-25 of it at -0.14, where 1 - 2^z is
// off by 2^-20.6 at most) and 2^z from o.
__device__ __forceinline__ float decay(float z, float *o) {
    float p = fmaf(z, -1.33335581e-3f, -9.61812911e-3f);
    p = fmaf(z, p, -5.55041087e-2f);
    p = fmaf(z, p, -2.40226507e-1f);
    p = fmaf(z, p, -6.93147181e-1f);
    const float e = __builtin_amdgcn_exp2f(z);
    const bool near = z > -0.14f;
    *o = near ? z * p : 1.0f - e;
    return near ? 1.0f - *o : e;
}

// V channels' rates, times log2(e); at any address (a few bytes, once a thread)
template <int V> __device__ __forceinline__ void load_rate(const float *p, float (&rate)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) rate[v] = p[v];
#pragma unroll
    for (int v = 0; v < V; ++v) rate[v] *= LOG2E;
}

// What a token's gate comes to.
struct Gate {
    float a, o;  // the decay, 1 - a
    float s;     // the input's scale
    float g, ng; // with a rate: sigma(r), 1 - sigma(r)
};

// Rates are >= 0, and come times log2(e). A closed gate (r = -infinity) gives a = 1, o = s = 0.
template <bool RATE> __device__ __forceinline__ Gate gate(float r, float rate2) {
    Gate k;
    if constexpr (RATE) {
        k.g = sigmoid2(r, &k.ng);
        k.a = decay(-rate2 * k.g, &k.o);
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
