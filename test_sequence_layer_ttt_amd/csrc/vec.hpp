// V consecutive elements of a storage type as fp32 values, in accesses of up
// to 16 bytes (V = 1: any alignment of the element).
#pragma once

#include "tile.hpp"

namespace ttt {

template <typename T, int V> struct VecIO;

template <> struct VecIO<float, 1> {
    typedef float Raw;
    static __device__ __forceinline__ Raw zero() { return 0.f; }
    static __device__ __forceinline__ Raw raw(const float *p) { return *p; }
    static __device__ __forceinline__ void unpack(Raw r, float (&x)[1]) { x[0] = r; }
    static __device__ __forceinline__ void store(float *p, const float (&x)[1]) { *p = x[0]; }
};
template <> struct VecIO<bf16_t, 1> {
    typedef bf16_t Raw;
    static __device__ __forceinline__ Raw zero() { return 0; }
    static __device__ __forceinline__ Raw raw(const bf16_t *p) { return *p; }
    static __device__ __forceinline__ void unpack(Raw r, float (&x)[1]) { x[0] = bf16_to_f32(r); }
    static __device__ __forceinline__ void store(bf16_t *p, const float (&x)[1]) { *p = f32_to_bf16(x[0]); }
};
template <> struct VecIO<float, 4> {
    typedef float4 Raw;
    static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
    static __device__ __forceinline__ Raw raw(const float *p) { return *reinterpret_cast<const float4 *>(p); }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[4]) {
        x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[4]) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <> struct VecIO<bf16_t, 4> {
    typedef uint2 Raw;
    static __device__ __forceinline__ Raw zero() { return make_uint2(0, 0); }
    static __device__ __forceinline__ Raw raw(const bf16_t *p) { return *reinterpret_cast<const uint2 *>(p); }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[4]) {
        x[0] = tile::lo_bf(r.x); x[1] = tile::hi_bf(r.x);
        x[2] = tile::lo_bf(r.y); x[3] = tile::hi_bf(r.y);
    }
    static __device__ __forceinline__ void store(bf16_t *p, const float (&x)[4]) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(tile::pack2(x[0], x[1]), tile::pack2(x[2], x[3]));
    }
};
template <> struct VecIO<float, 8> {
    struct Raw { float4 a, b; };
    static __device__ __forceinline__ Raw zero() {
        return {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    }
    static __device__ __forceinline__ Raw raw(const float *p) {
        const float4 *q = reinterpret_cast<const float4 *>(p);
        return {q[0], q[1]};
    }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[8]) {
        x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
        x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[8]) {
        float4 *q = reinterpret_cast<float4 *>(p);
        q[0] = make_float4(x[0], x[1], x[2], x[3]);
        q[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <> struct VecIO<bf16_t, 8> {
    typedef uint4 Raw;
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ Raw raw(const bf16_t *p) { return *reinterpret_cast<const uint4 *>(p); }
    static __device__ __forceinline__ void unpack(const Raw &r, float (&x)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = tile::lo_bf(w[i]);
            x[2 * i + 1] = tile::hi_bf(w[i]);
        }
    }
    static __device__ __forceinline__ void store(bf16_t *p, const float (&x)[8]) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(tile::pack2(x[0], x[1]), tile::pack2(x[2], x[3]),
                                                   tile::pack2(x[4], x[5]), tile::pack2(x[6], x[7]));
    }
};

template <typename T, int V>
__device__ __forceinline__ void vec_load(const T *p, float (&x)[V]) {
    VecIO<T, V>::unpack(VecIO<T, V>::raw(p), x);
}

// A store of 16 bytes that the chip's L2 need not keep: outputs larger than it, which only a
// later kernel reads.
template <typename T, int V> __device__ __forceinline__ void stream_store(T *p, const float (&x)[V]) {
    typedef __attribute__((ext_vector_type(4))) unsigned u4;
    if constexpr (V == 8 && sizeof(T) == 2) {
        const u4 v = {tile::pack2(x[0], x[1]), tile::pack2(x[2], x[3]), tile::pack2(x[4], x[5]), tile::pack2(x[6], x[7])};
        __builtin_nontemporal_store(v, reinterpret_cast<u4 *>(p));
    } else if constexpr (V == 4 && sizeof(T) == 4) {
        const u4 v = {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
        __builtin_nontemporal_store(v, reinterpret_cast<u4 *>(p));
    } else {
        VecIO<T, V>::store(p, x);
    }
}

// 1 / (1 + e^-s): e^-s overflows to infinity for very negative s and the
// quotient is then 0, which is the limit.
__device__ __forceinline__ float sigmoid_f(float s) { return __builtin_amdgcn_rcpf(1.0f + __expf(-s)); }

// e^x to about 1.5 steps of fp32: 2^t with t = x log2(e) rounded, times what
// the rounding and the constant's own tail leave, 1 + r ln 2 (r is below 2^-20
// for |x| < 10). Below -87 the result is 0 or a denormal and may be flushed.
__device__ __forceinline__ float exp_f(float x) {
    const float t = x * 1.44269504f;
    const float r = fmaf(x, 1.44269504f, -t) + x * 1.92596299e-8f;
    return __builtin_amdgcn_exp2f(t) * fmaf(r, 0.693147181f, 1.0f);
}

// x, or `low` where it is below that. A NaN stays one (fmax would return `low`).
template <typename T> __device__ __forceinline__ T at_least(T x, T low) { return x < low ? low : x; }

// log(1 + e^s) = max(s, 0) + log(1 + e), e = e^-|s| in (0, 1], which is
// 2 atanh(q), q = e / (2 + e) <= 1/3, by its series to q^15 (the next term is
// below 2^-26): small results keep their relative accuracy, about 2 steps.
__device__ __forceinline__ float softplus_f(float s) {
    const float e = exp_f(-fminf(fabsf(s), 100.f));
    const float q = e * __builtin_amdgcn_rcpf(2.0f + e), p = q * q;
    float c = fmaf(p, 1.0f / 15, 1.0f / 13);
    c = fmaf(p, c, 1.0f / 11);
    c = fmaf(p, c, 1.0f / 9);
    c = fmaf(p, c, 1.0f / 7);
    c = fmaf(p, c, 1.0f / 5);
    c = fmaf(p, c, 1.0f / 3);
    return (s <= 0.f ? 0.f : s) + 2.0f * fmaf(q * p, c, q);  // NaN stays NaN
}

}  // namespace ttt
