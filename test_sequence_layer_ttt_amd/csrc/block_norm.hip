// The seam between two blocks of a layer stack: the norm after a block, its
// gate, the residual sum and the norm before the next block.
//     n  = Norm(y) post_gamma (+ post_beta)
//     r' = scale resid + act(gate) n
//     x  = Norm(r') pre_gamma (+ pre_beta)
// with Norm(u) = u / sqrt(mean u^2 + eps) or (u - mean u) / sqrt(var u + eps).
//
// HBM bound: a row's resid, y and gate are read once, r' and x written once.
// TPR threads hold a row in registers (64: one wave a row, no barriers; 256:
// a workgroup a row), the statistics are sums of registers (of centred values,
// so a common offset of the row costs no digits), and the next row's loads
// are issued before this row's sums are waited for.
//
// The backward reads the same rows and the two outputs' gradients, forms the
// forward's values again in registers (nothing is saved by the forward), and
// keeps the per-column sums of the parameters' gradients in registers over
// all rows of a workgroup; column_sums joins the workgroups in a fixed order.
//     g  = dr' + rstd_r (h - [mean h] - rhat mean(h rhat)),  h = dx pre_gamma
//     dresid = scale g,   dgate = g n act',   dn = g act
//     dy = rstd_y (k - [mean k] - yhat mean(k yhat)),        k = dn post_gamma
// ([..]: with the mean's removal only).
#include "block.hpp"
#include "ttt.h"
#include "vec.hpp"

namespace ttt {
namespace {

constexpr int NT = 256;

__device__ __forceinline__ float wave_sum(float v) { return tile::rows4_sum(tile::row16_sum(v)); }

// Sum over the TPR threads of a row; every thread receives it. The LDS slots
// alternate from call to call, so one barrier a call is enough.
template <int TPR> struct RowSum {
    float (*red)[NT / 64];
    int slot = 0;
    __device__ __forceinline__ float operator()(float v) {
        v = wave_sum(v);
        if constexpr (TPR > 64) {
            red[slot][threadIdx.x / 64] = v;
            __syncthreads();
            v = (red[slot][0] + red[slot][1]) + (red[slot][2] + red[slot][3]);
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
            u = (red[slot][0] + red[slot][1]) + (red[slot][2] + red[slot][3]);
            v = (red[slot + 2][0] + red[slot + 2][1]) + (red[slot + 2][2] + red[slot + 2][3]);
            slot ^= 1;
        }
    }
};

// the gate's activation and its derivative
__device__ __forceinline__ void activate(int act, float g, float &a, float &da) {
    if (act == TTT_ACT_SIGMOID) {
        a = sigmoid_f(g);
        da = a * (1.f - a);
    } else if (act == TTT_ACT_SILU) {
        const float s = sigmoid_f(g);
        a = g * s;
        da = s * fmaf(g, 1.f - s, 1.f);
    } else if (act == TTT_ACT_TANH) {
        a = tanhf(g);
        da = 1.f - a * a;
    } else {
        a = g;
        da = 1.f;
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

// One row's inputs, fetched ahead
template <class C, typename TIO, typename TR> struct RowIn {
    typename C::template Raws<TR> resid;
    typename C::template Raws<TIO> y, gate;
    bool live;
};

template <int TPR, int VEC, int NV, typename TIO, typename TR>
__global__ __launch_bounds__(NT) void block_norm_fwd(NormArgs a, int rows) {
    typedef Cols<TPR, VEC, NV> C;
    constexpr int E = C::E, RPW = NT / TPR;
    constexpr bool HOLD = E <= 16;  // parameters in registers over all rows
    __shared__ float red[4][NT / 64];
    RowSum<TPR> sum{red};
    const C c{a.D, static_cast<int>(threadIdx.x % TPR)};
    const float inv_d = 1.0f / static_cast<float>(a.D);
    const int step = gridDim.x * RPW;
    float pg[E], pb[E], qg[E], qb[E], sc[E];
    if constexpr (HOLD) {
        c.param(a.post_gamma, 1.f, pg);
        c.param(a.post_beta, 0.f, pb);
        c.param(a.pre_gamma, 1.f, qg);
        c.param(a.pre_beta, 0.f, qb);
        c.param(a.scale, 1.f, sc);
    }
    auto fetch = [&](int row, RowIn<C, TIO, TR> &in) {
        const int b = row / a.L, t = row - b * a.L;
        in.live = !a.lens || t < a.lens[b];
        if (!in.live) return;
        c.fetch(static_cast<const TR *>(a.resid) + b * a.rb + t * a.rt, in.resid);
        c.fetch(static_cast<const TIO *>(a.y) + b * a.yb + t * a.yt, in.y);
        if (a.gmode == TTT_GATE_TOKEN) c.fetch(static_cast<const TIO *>(a.gate) + b * a.gb + t * a.gt, in.gate);
    };
    int row = blockIdx.x * RPW + threadIdx.x / TPR;
    RowIn<C, TIO, TR> in;
    if (row < rows) fetch(row, in);
    for (; row < rows; row += step) {
        TR *ro = static_cast<TR *>(a.resid_out) + static_cast<int64_t>(row) * a.D;
        TIO *xo = static_cast<TIO *>(a.x) + static_cast<int64_t>(row) * a.D;
        const bool live = in.live;
        float n[E], r[E], g[E];
        if (live) {
            c.unpack(in.y, n);
            c.unpack(in.resid, r);
            if (a.gmode == TTT_GATE_TOKEN) c.unpack(in.gate, g);
        }
        if (row < rows - step) fetch(row + step, in);
        if (!live) {  // past the sequence's end: zeros
#pragma unroll
            for (int e = 0; e < E; ++e) n[e] = 0.f;
            c.store(ro, n);
            c.store(xo, n);
            continue;
        }
        if (a.gmode == TTT_GATE_CHANNEL) c.load(static_cast<const float *>(a.gate), g);
        if (a.gmode == TTT_GATE_SEQUENCE)
            c.load(static_cast<const float *>(a.gate) + static_cast<int64_t>(row / a.L) * a.D, g);
        c.hat(n, a.layer, a.eps, inv_d, sum);
        if constexpr (!HOLD) {
            c.param(a.post_gamma, 1.f, pg);
            c.param(a.post_beta, 0.f, pb);
            c.param(a.scale, 1.f, sc);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            n[e] = fmaf(n[e], pg[e], pb[e]);
            if (a.gmode != TTT_GATE_NONE) {
                float v, dv;
                activate(a.act, g[e], v, dv);
                n[e] *= v;
            }
            r[e] = fmaf(sc[e], r[e], n[e]);
        }
        c.store(ro, r);
        c.hat(r, a.layer, a.eps, inv_d, sum);
        if constexpr (!HOLD) {
            c.param(a.pre_gamma, 1.f, qg);
            c.param(a.pre_beta, 0.f, qb);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = fmaf(r[e], qg[e], qb[e]);
        c.store(xo, r);
    }
}

// column quantities of the backward's partials
enum { Q_POST_G, Q_PRE_G, Q_SCALE, Q_POST_B, Q_PRE_B, Q_GATE, Q_N };

template <int TPR, int VEC, int NV, typename TIO, typename TR>
__global__ __launch_bounds__(NT) void block_norm_bwd(NormBwdArgs ga) {
    typedef Cols<TPR, VEC, NV> C;
    constexpr int E = C::E, RPW = NT / TPR;
    __shared__ float red[4][NT / 64];
    __shared__ float comb[RPW > 1 ? RPW * TPR * E : 1];
    const NormArgs &a = ga.f;
    RowSum<TPR> sum{red};
    const C c{a.D, static_cast<int>(threadIdx.x % TPR)};
    const float inv_d = 1.0f / static_cast<float>(a.D);
    // rows of this workgroup: with a gate for each sequence those of sequence
    // blockIdx.y, else of the whole batch
    const int rows = a.gmode == TTT_GATE_SEQUENCE ? a.L : a.B * a.L;
    const int row0 = a.gmode == TTT_GATE_SEQUENCE ? blockIdx.y * a.L : 0;
    const int step = gridDim.x * RPW;
    float acc[Q_N][E] = {};
    for (int i = blockIdx.x * RPW + threadIdx.x / TPR; i < rows; i += step) {
        const int row = row0 + i;
        const int b = row / a.L, t = row - b * a.L;
        const int64_t at = static_cast<int64_t>(row) * a.D;
        float u[E], v[E], w[E];
        if (a.lens && t >= a.lens[b]) {  // past the sequence's end: zeros, nothing read
#pragma unroll
            for (int e = 0; e < E; ++e) u[e] = 0.f;
            c.store(static_cast<TR *>(ga.dresid) + at, u);
            c.store(static_cast<TIO *>(ga.dy) + at, u);
            if (a.gmode == TTT_GATE_TOKEN) c.store(static_cast<TIO *>(ga.dgate) + at, u);
            continue;
        }
        float yh[E], res[E], g[E], dxv[E], dro[E];
        c.load(static_cast<const TIO *>(a.y) + b * a.yb + t * a.yt, yh);
        c.load(static_cast<const TR *>(a.resid) + b * a.rb + t * a.rt, res);
        c.load(static_cast<const TIO *>(ga.dx) + at, dxv);
        c.load(static_cast<const TR *>(ga.dresid_out) + at, dro);
        if (a.gmode == TTT_GATE_TOKEN) c.load(static_cast<const TIO *>(a.gate) + b * a.gb + t * a.gt, g);
        if (a.gmode == TTT_GATE_CHANNEL) c.load(static_cast<const float *>(a.gate), g);
        if (a.gmode == TTT_GATE_SEQUENCE) c.load(static_cast<const float *>(a.gate) + static_cast<int64_t>(b) * a.D, g);
        const float yr = c.hat(yh, a.layer, a.eps, inv_d, sum);
        // u: r', then its normalised value; w: the norm after the block
        c.param(a.post_gamma, 1.f, v);
        c.param(a.post_beta, 0.f, w);
        c.param(a.scale, 1.f, u);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            w[e] = fmaf(yh[e], v[e], w[e]);
            float x = 1.f, dv;
            if (a.gmode != TTT_GATE_NONE) activate(a.act, g[e], x, dv);
            u[e] = fmaf(u[e], res[e], x * w[e]);
        }
        const float rr = c.hat(u, a.layer, a.eps, inv_d, sum);
        c.param(a.pre_gamma, 1.f, v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            acc[Q_PRE_G][e] = fmaf(dxv[e], u[e], acc[Q_PRE_G][e]);
            acc[Q_PRE_B][e] += dxv[e];
            dxv[e] *= v[e];
        }
        c.unhat(dxv, u, rr, a.layer, inv_d, sum);
        c.param(a.scale, 1.f, v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            dro[e] += dxv[e];
            acc[Q_SCALE][e] = fmaf(dro[e], res[e], acc[Q_SCALE][e]);
            u[e] = dro[e] * v[e];
        }
        c.store(static_cast<TR *>(ga.dresid) + at, u);
        c.param(a.post_gamma, 1.f, v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float dn = dro[e];
            if (a.gmode != TTT_GATE_NONE) {
                float x, dv;
                activate(a.act, g[e], x, dv);
                u[e] = dn * w[e] * dv;
                dn *= x;
            }
            acc[Q_POST_G][e] = fmaf(dn, yh[e], acc[Q_POST_G][e]);
            acc[Q_POST_B][e] += dn;
            w[e] = dn * v[e];
        }
        if (a.gmode == TTT_GATE_TOKEN) {
            c.store(static_cast<TIO *>(ga.dgate) + at, u);
        } else if (a.gmode != TTT_GATE_NONE) {
#pragma unroll
            for (int e = 0; e < E; ++e) acc[Q_GATE][e] += u[e];
        }
        c.unhat(w, yh, yr, a.layer, inv_d, sum);
        c.store(static_cast<TIO *>(ga.dy) + at, w);
    }
    float *part = ga.ws + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * Q_N * a.D;
    const bool want[Q_N] = {ga.dpost_gamma != nullptr, ga.dpre_gamma != nullptr, ga.dscale != nullptr,
                            ga.dpost_beta != nullptr, ga.dpre_beta != nullptr,
                            a.gmode == TTT_GATE_CHANNEL || a.gmode == TTT_GATE_SEQUENCE};
#pragma unroll
    for (int q = 0; q < Q_N; ++q) {
        if (!want[q]) continue;
        if constexpr (RPW > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e) comb[(e * RPW + threadIdx.x / TPR) * TPR + c.i] = acc[q][e];
            __syncthreads();
            if (threadIdx.x < TPR) {
                float s[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    s[e] = 0.f;
#pragma unroll
                    for (int k = 0; k < RPW; ++k) s[e] += comb[(e * RPW + k) * TPR + c.i];
                }
                c.store(part + static_cast<int64_t>(q) * a.D, s);
            }
        } else {
            c.store(part + static_cast<int64_t>(q) * a.D, acc[q]);
        }
    }
}

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool vec_ok(const NormArgs &a, int v) {
    return a.D % v == 0 && a.rb % v == 0 && a.rt % v == 0 && a.yb % v == 0 && a.yt % v == 0 &&
           a.gb % v == 0 && a.gt % v == 0 && aligned(a.resid, 16) && aligned(a.y, 16) &&
           aligned(a.gate, 16) && aligned(a.post_gamma, 16) && aligned(a.post_beta, 16) &&
           aligned(a.pre_gamma, 16) && aligned(a.pre_beta, 16) && aligned(a.scale, 16);
}

template <int TPR, int VEC, int NV, typename TIO, typename TR> struct Fwd {
    static hipError_t run(const NormArgs &a, hipStream_t s) {
        const int rows = a.B * a.L, rpw = NT / TPR;
        const int64_t need = (static_cast<int64_t>(rows) + rpw - 1) / rpw;
        const int grid = static_cast<int>(need < 2048 ? need : 2048);
        hipLaunchKernelGGL((block_norm_fwd<TPR, VEC, NV, TIO, TR>), dim3(grid), dim3(NT), 0, s, a, rows);
        return hipGetLastError();
    }
};

template <int TPR, int VEC, int NV, typename TIO, typename TR> struct Bwd {
    static hipError_t run(const NormBwdArgs &g, hipStream_t s) {
        const NormArgs &a = g.f;
        int64_t groups;
        int nq;
        block_norm_backward_partials(a.B, a.L, a.D, a.gmode, &groups, &nq);
        const int outer = a.gmode == TTT_GATE_SEQUENCE ? a.B : 1;
        hipLaunchKernelGGL((block_norm_bwd<TPR, VEC, NV, TIO, TR>), dim3(static_cast<unsigned>(groups / outer), outer),
                           dim3(NT), 0, s, g);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        ColumnSums c{g.ws, static_cast<int64_t>(nq) * a.D, static_cast<int>(groups)};
        const int64_t D = a.D;
        c.add(Q_POST_G * D, a.D, 1, g.dpost_gamma);
        c.add(Q_PRE_G * D, a.D, 1, g.dpre_gamma);
        c.add(Q_SCALE * D, a.D, 1, g.dscale);
        c.add(Q_POST_B * D, a.D, 1, g.dpost_beta);
        c.add(Q_PRE_B * D, a.D, 1, g.dpre_beta);
        if (a.gmode == TTT_GATE_CHANNEL || a.gmode == TTT_GATE_SEQUENCE)
            c.add(Q_GATE * D, a.D, outer, static_cast<float *>(g.dgate));
        return launch_column_sums(c, s);
    }
};

// A row of up to 1024 columns is one wave's (no barriers), a longer one a
// workgroup's. Columns go in vectors of 4 (8 for the forward's long rows),
// one by one where the width or an address does not allow vectors.
template <template <int, int, int, typename, typename> class K, int WIDE, typename TIO, typename TR, typename A>
hipError_t by_width(const A &a, int D, bool vec4, bool wide, hipStream_t s) {
    if (vec4 && D <= 1024) {
        if (D <= 256) return K<64, 4, 1, TIO, TR>::run(a, s);
        if (D <= 512) return K<64, 4, 2, TIO, TR>::run(a, s);
        if (D <= 768) return K<64, 4, 3, TIO, TR>::run(a, s);
        return K<64, 4, 4, TIO, TR>::run(a, s);
    }
    if (wide && vec4) {
        if (D <= 2048) return K<256, WIDE, 8 / WIDE, TIO, TR>::run(a, s);
        if (D <= 4096) return K<256, WIDE, 16 / WIDE, TIO, TR>::run(a, s);
        return K<256, WIDE, 32 / WIDE, TIO, TR>::run(a, s);
    }
    if (D <= 256) return K<64, 1, 4, TIO, TR>::run(a, s);
    if (D <= 1024) return K<64, 1, 16, TIO, TR>::run(a, s);
    if (D <= 4096) return K<256, 1, 16, TIO, TR>::run(a, s);
    return K<256, 1, 32, TIO, TR>::run(a, s);
}

template <template <int, int, int, typename, typename> class K, int WIDE, typename A>
hipError_t by_type(const A &a, const NormArgs &f, bool vec4, bool wide, hipStream_t s) {
    if (f.io == TTT_F32) return by_width<K, WIDE, float, float>(a, f.D, vec4, wide, s);
    return f.rio == TTT_F32 ? by_width<K, WIDE, bf16_t, float>(a, f.D, vec4, wide, s)
                            : by_width<K, WIDE, bf16_t, bf16_t>(a, f.D, vec4, wide, s);
}

}  // namespace

hipError_t launch_block_norm(const NormArgs &a, hipStream_t stream) {
    const bool out = aligned(a.resid_out, 16) && aligned(a.x, 16);
    return by_type<Fwd, 8>(a, a, out && vec_ok(a, 4), out && vec_ok(a, 8), stream);
}

void block_norm_backward_partials(int B, int L, int D, int gmode, int64_t *groups, int *quantities) {
    const int rpw = D <= 1024 ? NT / 64 : 1;  // rows a workgroup holds at a time
    const int64_t outer = gmode == TTT_GATE_SEQUENCE ? B : 1;
    const int64_t rows = gmode == TTT_GATE_SEQUENCE ? L : static_cast<int64_t>(B) * L;
    int64_t per = (rows + rpw - 1) / rpw;
    const int64_t most = outer < 512 ? 512 / outer : 1;
    if (per > most) per = most;
    if (per < 1) per = 1;
    *groups = outer * per > 0 ? outer * per : 1;
    *quantities = Q_N;
}

hipError_t launch_block_norm_backward(const NormBwdArgs &g, hipStream_t stream) {
    const bool out = aligned(g.dresid_out, 16) && aligned(g.dx, 16) && aligned(g.dresid, 16) &&
                     aligned(g.dy, 16) && aligned(g.dgate, 16) && aligned(g.ws, 16);
    const bool v = out && vec_ok(g.f, 4);
    return by_type<Bwd, 4>(g, g.f, v, v, stream);
}

}  // namespace ttt
