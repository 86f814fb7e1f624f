// Rows of the block norm in registers: the columns of a thread, their loads and
// stores, the sums over a row and the norms, and the choice of a kernel by
// width and types (block_norm.hip, block_norm_bwd.hip).
#pragma once

#include "block.hpp"
#include "ttt.h"
#include "vec.hpp"

namespace ttt {
namespace norm {

// threads of a workgroup: four rows of 64, or one row
constexpr int threads(int tpr) { return tpr > 256 ? tpr : 256; }

__device__ __forceinline__ float wave_sum(float v) { return tile::rows4_sum(tile::row16_sum(v)); }

// Sum over the TPR threads of a row; every thread receives it. The LDS slots
// alternate from call to call, so one barrier a call is enough.
template <int TPR> struct RowSum {
    static constexpr int NW = threads(TPR) / 64;
    float (*red)[NW];
    int slot = 0;
    __device__ __forceinline__ static float over_waves(const float (&p)[NW]) {
        float s = (p[0] + p[1]) + (p[2] + p[3]);
#pragma unroll
        for (int k = 4; k < NW; k += 4) s += (p[k] + p[k + 1]) + (p[k + 2] + p[k + 3]);
        return s;
    }
    __device__ __forceinline__ float operator()(float v) {
        v = wave_sum(v);
        if constexpr (TPR > 64) {
            red[slot][threadIdx.x / 64] = v;
            __syncthreads();
            v = over_waves(red[slot]);
            slot ^= 1;
        }
        return v;
    }
    __device__ __forceinline__ void two(float &u, float &v) {
        u = wave_sum(u);
        v = wave_sum(v);
        if constexpr (TPR > 64) {
            red[slot][threadIdx.x / 64] = u;
            red[slot + 2][threadIdx.x / 64] = v;
            __syncthreads();
            u = over_waves(red[slot]);
            v = over_waves(red[slot + 2]);
            slot ^= 1;
        }
    }
};

// the gate's activation and its derivative, one choice for all of a row's values
template <int E> __device__ __forceinline__ void activate(int act, const float (&g)[E], float (&a)[E], float (&da)[E]) {
    if (act == TTT_ACT_SIGMOID) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            a[e] = sigmoid_f(g[e]);
            da[e] = a[e] * (1.f - a[e]);
        }
    } else if (act == TTT_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float s = sigmoid_f(g[e]);
            a[e] = g[e] * s;
            da[e] = s * fmaf(g[e], 1.f - s, 1.f);
        }
    } else if (act == TTT_ACT_TANH) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            a[e] = tanhf(g[e]);
            da[e] = 1.f - a[e] * a[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            a[e] = g[e];
            da[e] = 1.f;
        }
    }
}

// The columns of one thread: NV vectors of VEC, TPR vectors apart.
template <int TPR, int VEC, int NV> struct Cols {
    static constexpr int E = VEC * NV;
    int D, i;
    __device__ __forceinline__ int col(int j) const { return (j * TPR + i) * VEC; }
    __device__ __forceinline__ bool in(int j) const { return col(j) < D; }

    template <typename T> struct Raws {
        typename VecIO<T, VEC>::Raw r[NV];
    };
    template <typename T> __device__ __forceinline__ void fetch(const T *p, Raws<T> &r) const {
#pragma unroll
        for (int j = 0; j < NV; ++j) r.r[j] = in(j) ? VecIO<T, VEC>::raw(p + col(j)) : VecIO<T, VEC>::zero();
    }
    template <typename T> __device__ __forceinline__ void unpack(const Raws<T> &r, float (&x)[E]) const {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float v[VEC];
            VecIO<T, VEC>::unpack(r.r[j], v);
#pragma unroll
            for (int k = 0; k < VEC; ++k) x[j * VEC + k] = v[k];
        }
    }
    template <typename T> __device__ __forceinline__ void load(const T *p, float (&x)[E]) const {
        Raws<T> r;
        fetch(p, r);
        unpack(r, x);
    }
    // a parameter row, `other` where there is none; 0 past the row's end
    __device__ __forceinline__ void param(const float *p, float other, float (&x)[E]) const {
        if (p) {
            load(p, x);
            return;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = in(e / VEC) ? other : 0.f;
    }
    template <typename T> __device__ __forceinline__ void store(T *p, const float (&x)[E]) const {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!in(j)) continue;
            float v[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[k] = x[j * VEC + k];
            VecIO<T, VEC>::store(p + col(j), v);
        }
    }
    // u <- (u - [mean]) rstd, 0 past the row's end
    __device__ __forceinline__ float hat(float (&u)[E], int layer, float eps, float inv_d,
                                         RowSum<TPR> &sum) const {
        if (layer) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s += u[e];
            const float m = sum(s) * inv_d;
#pragma unroll
            for (int e = 0; e < E; ++e) u[e] = in(e / VEC) ? u[e] - m : 0.f;
        }
        float v = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) v = fmaf(u[e], u[e], v);
        const float rstd = rsqrtf(sum(v) * inv_d + eps);
#pragma unroll
        for (int e = 0; e < E; ++e) u[e] *= rstd;
        return rstd;
    }
    // h <- rstd (h - [mean h] - hat mean(h hat))
    __device__ __forceinline__ void unhat(float (&h)[E], const float (&hat)[E], float rstd, int layer,
                                          float inv_d, RowSum<TPR> &sum) const {
        float s = 0.f, p = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            s += h[e];
            p = fmaf(h[e], hat[e], p);
        }
        sum.two(s, p);
        s = layer ? s * inv_d : 0.f;
        p *= inv_d;
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = rstd * (h[e] - s - hat[e] * p);
    }
};

inline bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline bool vec_ok(const NormArgs &a, int v) {
    return a.D % v == 0 && a.rb % v == 0 && a.rt % v == 0 && a.yb % v == 0 && a.yt % v == 0 &&
           a.gb % v == 0 && a.gt % v == 0 && aligned(a.resid, 16) && aligned(a.y, 16) &&
           aligned(a.gate, 16) && aligned(a.post_gamma, 16) && aligned(a.post_beta, 16) &&
           aligned(a.pre_gamma, 16) && aligned(a.pre_beta, 16) && aligned(a.scale, 16);
}

// A row of up to 1024 columns is one wave's (no barriers), a longer one a
// workgroup's. Columns go in vectors of 4 (8 for the forward's long rows),
// one by one where the width or an address does not allow vectors. The backward
// (BWD) holds seven values and up to six sums of a column in registers: eight
// columns of a thread are two waves a SIMD, so its rows of 2049 to 4096 columns
// go to 512 threads (D = 2560, 2457 rows: 47 us, 54 with sixteen columns; D =
// 4096, 1536 rows: 42 and 44). Longer rows spill either way and stay with 256,
// which may spill to more registers (D = 8192 with betas: 150 us, 169 with 512).
template <template <int, int, int, typename, typename> class K, int WIDE, bool BWD, typename TIO, typename TR, typename A>
hipError_t by_width(const A &a, int D, bool vec4, bool wide, hipStream_t s) {
    if (vec4 && D <= 1024) {
        if (D <= 256) return K<64, 4, 1, TIO, TR>::run(a, s);
        if (D <= 512) return K<64, 4, 2, TIO, TR>::run(a, s);
        if (D <= 768) return K<64, 4, 3, TIO, TR>::run(a, s);
        return K<64, 4, 4, TIO, TR>::run(a, s);
    }
    if (wide && vec4) {
        if (D <= 2048) return K<256, WIDE, 8 / WIDE, TIO, TR>::run(a, s);
        if (D <= 4096) return K<BWD ? 512 : 256, WIDE, (BWD ? 8 : 16) / WIDE, TIO, TR>::run(a, s);
        return K<256, WIDE, 32 / WIDE, TIO, TR>::run(a, s);
    }
    if (D <= 256) return K<64, 1, 4, TIO, TR>::run(a, s);
    if (D <= 1024) return K<64, 1, 16, TIO, TR>::run(a, s);
    if (D <= 4096) return K<256, 1, 16, TIO, TR>::run(a, s);
    return K<256, 1, 32, TIO, TR>::run(a, s);
}

template <template <int, int, int, typename, typename> class K, int WIDE, bool BWD, typename A>
hipError_t by_type(const A &a, const NormArgs &f, bool vec4, bool wide, hipStream_t s) {
    if (f.io == TTT_F32) return by_width<K, WIDE, BWD, float, float>(a, f.D, vec4, wide, s);
    return f.rio == TTT_F32 ? by_width<K, WIDE, BWD, bf16_t, float>(a, f.D, vec4, wide, s)
                            : by_width<K, WIDE, BWD, bf16_t, bf16_t>(a, f.D, vec4, wide, s);
}

}  // namespace norm
}  // namespace ttt
