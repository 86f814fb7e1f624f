// Rows of fp32 or bf16 in 8 bits: scale = max |x| / 127 in fp32 and
// q = x / scale rounded to the nearest whole number, ties to even, of the
// exact quotient, held to -127 .. 127.
//
// The quotient is not divided out: q0 = rint(x rcp(scale)) is the nearest
// whole number or one beside it, r = x - q0 scale is exact in one fused step
// (where |x| >= scale both are multiples of scale's last place; where it is
// not, q0 is 0 or r is a difference of numbers within a factor of two), and
// r against scale / 2 says which. Scales below 2^-120, where the reciprocal or
// the half could leave fp32's range, are divided in 64 bits.
//
// A row that holds an infinity or a NaN has a NaN for its scale and zeros for
// q, so that its products are NaN.
#pragma once

#include "i8.hpp"

#include <math.h>

namespace ttt {

struct Scale {
    float s, inv, half;
    bool finite, normal;
    // from the bits of the row's largest |x|
    __device__ __forceinline__ explicit Scale(uint32_t most) {
        finite = most < 0x7f800000u;
        s = finite ? __uint_as_float(most) / 127.0f : __uint_as_float(0x7fc00000u);
        normal = s >= 0x1p-120f;
        inv = __builtin_amdgcn_rcpf(s);
        half = 0.5f * s;
    }
    __device__ __forceinline__ int nearest(float x) const {
        if (normal) {
            float q = __builtin_rintf(x * inv);
            const float r = fmaf(-q, s, x);
            const bool odd = static_cast<int>(q) & 1;
            if (r > half || (r == half && odd)) q += 1.0f;
            if (r < -half || (r == -half && odd)) q -= 1.0f;
            return static_cast<int>(fminf(fmaxf(q, -127.0f), 127.0f));
        }
        if (!(s > 0.f)) return 0;  // a row of zeros, or one that is not finite
        const double q = __builtin_rint(static_cast<double>(x) / static_cast<double>(s));
        return static_cast<int>(fmin(fmax(q, -127.0), 127.0));
    }
    // V values to bytes at q. Nearly always rint's whole number is the nearest and no tie, which
    // |r| < half says of all V at once.
    template <int V> __device__ __forceinline__ void put(const float (&x)[V], int8_t *q) const {
        int p[V];
        bool plain = true;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float f = __builtin_rintf(x[e] * inv);
            plain = plain && fabsf(fmaf(-f, s, x[e])) < half;
            p[e] = static_cast<int>(f);
        }
        if (!(plain && normal)) {
#pragma unroll
            for (int e = 0; e < V; ++e) p[e] = nearest(x[e]);
        }
        if constexpr (V == 1) {
            q[0] = static_cast<int8_t>(p[0]);
        } else {
            uint32_t w[V / 4];
#pragma unroll
            for (int e = 0; e < V / 4; ++e)
                w[e] = (p[4 * e] & 255) | (p[4 * e + 1] & 255) << 8 | (p[4 * e + 2] & 255) << 16 |
                       static_cast<uint32_t>(p[4 * e + 3]) << 24;
            if constexpr (V == 4)
                *reinterpret_cast<uint32_t *>(q) = w[0];
            else
                *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
        }
    }
};

}  // namespace ttt
