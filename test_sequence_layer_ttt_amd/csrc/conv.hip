// Short causal convolution of [B,L,C] features (a block's input, or columns of a
// projection's output), one filter of K = 2..4 taps for each channel:
//     z_t = bias + sum_k w_k x_{t-K+1+k},   y_t = z_t or z_t sigma(z_t),
// where the K - 1 tokens before the first come from a state (or are zero) and
// the last K - 1 tokens of each sequence are its state afterwards.
//
//  conv_fwd   HBM bound: x is read once and y written once. A thread holds V
//             consecutive channels (16 bytes) and walks over T tokens with the
//             last K - 1 of them in registers, so a token is read again only
//             at the T-token borders (from the chip's caches). Rows are loaded
//             U at a time, while the U before are worked on.
//             B=2 L=8192 C=2176 bf16: 31.7 us, 4.5 TB/s (a plain copy: 4.8).
//  conv_step  one token: the state is read, shifted and written in place.
//             B=64 C=2176: 2.3 MB in 4.4 us, which is a launch's own time.
//  conv_bwd   with g_t = dy_t act'(z_t):
//                 dx_t = sum_k w_k g_{t+K-1-k},   dw_k = sum_t g_t x_{t-K+1+k}.
//             The same walk with z_t formed again (x and dy read once, dx
//             written once); dw and db are summed over a workgroup's tokens in
//             registers and LDS and over the workgroups by column_sums, in a
//             fixed order. B=4 L=2048 C=896 bf16: 19.4 us for 44 MB. 52 vector
//             instructions a value (2.4 of them transcendental) are 12.6 us on
//             the compute units that hold two of the 448 workgroups; they hold
//             the vector units 64 % of the time, waves wait 40 % of theirs: for
//             their first rows, and for LDS in the K + 1 sums at the end.
#include "block.hpp"
#include "vec.hpp"

namespace ttt {
namespace {

constexpr int NT = 256;

// a row of (state, x): row i < K - 1 is the state's row i, row i >= K - 1 is
// token i - (K - 1)
template <int K, int V, typename T>
__device__ __forceinline__ typename VecIO<T, V>::Raw full_row(const T *x, int64_t xt, const T *st, int C,
                                                              int i) {
    if (i >= K - 1) return VecIO<T, V>::raw(x + static_cast<int64_t>(i - (K - 1)) * xt);
    return st ? VecIO<T, V>::raw(st + static_cast<int64_t>(i) * C) : VecIO<T, V>::zero();
}

template <int K, int V>
__device__ __forceinline__ void load_weights(const float *w, const float *bias, int c, float (&wk)[K][V],
                                             float (&bv)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bv[v] = bias ? bias[c + v] : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) wk[k][v] = w[static_cast<int64_t>(c + v) * K + k];
    }
}

template <int K, int V, typename T>
__global__ __launch_bounds__(NT) void conv_fwd(ConvArgs a, int tokens) {
    typedef VecIO<T, V> IO;
    constexpr int U = 4;
    const int c = (blockIdx.y * NT + threadIdx.x) * V;
    if (c >= a.C) return;
    const int b = blockIdx.z, t0 = blockIdx.x * tokens;
    const int t1 = min(t0 + tokens, a.L);
    const int n = a.lens ? max(0, min(a.lens[b], a.L)) : a.L;
    const T *x = static_cast<const T *>(a.x) + static_cast<int64_t>(b) * a.xb + c;
    const T *st = a.state ? static_cast<const T *>(a.state) + static_cast<int64_t>(b) * (K - 1) * a.C + c : nullptr;
    T *y = a.L ? static_cast<T *>(a.y) + static_cast<int64_t>(b) * a.yb + c : nullptr;
    float wk[K][V], bv[V], win[K][V];
    load_weights<K, V>(a.w, a.bias, c, wk, bv);
    const int te = min(t1, n);  // tokens past the sequence's end are not read
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
        if (t0 < te) IO::unpack(full_row<K, V>(x, a.xt, st, a.C, t0 + k), win[k]);
    }
    typename IO::Raw next[U];
    auto fetch = [&](int t) {
#pragma unroll
        for (int u = 0; u < U; ++u) next[u] = IO::raw(x + static_cast<int64_t>(min(t + u, te - 1)) * a.xt);
    };
    if (t0 < te) fetch(t0);
    for (int t = t0; t < te; t += U) {
        typename IO::Raw r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = next[u];
        if (t + U < te) fetch(t + U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            IO::unpack(r[u], win[K - 1]);
            float z[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                z[v] = bv[v];
#pragma unroll
                for (int k = 0; k < K; ++k) z[v] = fmaf(wk[k][v], win[k][v], z[v]);
                if (a.silu) z[v] *= sigmoid_f(z[v]);
            }
            if (t + u < te) IO::store(y + static_cast<int64_t>(t + u) * a.yt, z);
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) win[k][v] = win[k + 1][v];
        }
    }
    float zero[V] = {};
    for (int t = max(t0, n); t < t1; ++t) IO::store(y + static_cast<int64_t>(t) * a.yt, zero);
    // the state after token n - 1: rows n .. n + K - 2 of (state, x). All rows
    // are read before any is written (state_out may be the state itself).
    if (a.state_out && blockIdx.x == 0) {
        T *so = static_cast<T *>(a.state_out) + static_cast<int64_t>(b) * (K - 1) * a.C + c;
        typename IO::Raw r[K - 1];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) r[j] = full_row<K, V>(x, a.xt, st, a.C, n + j);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            float v[V];
            IO::unpack(r[j], v);
            IO::store(so + static_cast<int64_t>(j) * a.C, v);
        }
    }
}

template <int K, int V, typename T>
__global__ __launch_bounds__(NT) void conv_step(ConvArgs a) {
    typedef VecIO<T, V> IO;
    const int vecs = a.C / V;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * NT + threadIdx.x;
    if (i >= static_cast<int64_t>(a.B) * vecs) return;
    const int64_t b = i / vecs;
    const int c = static_cast<int>(i % vecs) * V;
    T *st = static_cast<T *>(a.state_out) + b * (K - 1) * a.C + c;
    typename IO::Raw r[K];
#pragma unroll
    for (int k = 0; k < K - 1; ++k) r[k] = IO::raw(st + static_cast<int64_t>(k) * a.C);
    r[K - 1] = IO::raw(static_cast<const T *>(a.x) + b * a.xb + c);
    float wk[K][V], z[V];
    load_weights<K, V>(a.w, a.bias, c, wk, z);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float v[V];
        IO::unpack(r[k], v);
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] = fmaf(wk[k][e], v[e], z[e]);
        if (k) IO::store(st + static_cast<int64_t>(k - 1) * a.C, v);
    }
    if (a.silu) {
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] *= sigmoid_f(z[e]);
    }
    IO::store(static_cast<T *>(a.y) + b * a.yb + c, z);
}

constexpr int BT = 16;             // tokens a thread of conv_bwd walks over
constexpr int BC = 32;             // channel vectors of a workgroup
constexpr int BR = NT / BC;        // token runs of a workgroup

template <int K, int V, typename T>
__global__ __launch_bounds__(NT) void conv_bwd(ConvBwdArgs g) {
    typedef VecIO<T, V> IO;
    constexpr int U = 4;
    __shared__ float red[BR][BC * V];
    const ConvArgs &a = g.f;
    const int lane = threadIdx.x % BC, run = threadIdx.x / BC;
    const int c = (blockIdx.y * BC + lane) * V;
    const bool live = c < a.C;
    const int b = blockIdx.z, t0 = (blockIdx.x * BR + run) * BT;
    const int n = a.lens ? max(0, min(a.lens[b], a.L)) : a.L;
    float dw[K][V] = {}, db[V] = {};
    // dx rows are emitted K - 1 tokens behind the walk; the first run also
    // emits the K - 1 rows of the state (tokens -(K-1) .. -1)
    if (live && (t0 < a.L || t0 == 0)) {
        const T *x = static_cast<const T *>(a.x) + static_cast<int64_t>(b) * a.xb + c;
        const T *dy = static_cast<const T *>(g.dy) + static_cast<int64_t>(b) * g.dyb + c;
        T *dx = static_cast<T *>(g.dx) + static_cast<int64_t>(b) * g.dxb + c;
        const int64_t so = static_cast<int64_t>(b) * (K - 1) * a.C + c;
        const T *st = a.state ? static_cast<const T *>(a.state) + so : nullptr;
        const T *dso = g.dstate_out ? static_cast<const T *>(g.dstate_out) + so : nullptr;
        T *ds = g.dstate ? static_cast<T *>(g.dstate) + so : nullptr;
        float wk[K][V], bv[V], win[K][V] = {}, gw[K][V] = {};
        load_weights<K, V>(a.w, a.bias, c, wk, bv);
        if (t0 < n) {
#pragma unroll
            for (int k = 0; k < K - 1; ++k) IO::unpack(full_row<K, V>(x, a.xt, st, a.C, t0 + k), win[k]);
        }
        const int t1 = min(t0 + BT, a.L);   // dx rows t0 .. t1 - 1 are this thread's
        const int te = t1 + K - 1;          // the walk
        const int tn = min(te, n) - 1;      // the last row that is read
        typename IO::Raw nx[U], nd[U];
        auto fetch = [&](int t) {  // rows behind the last are read from it and count as zeros
#pragma unroll
            for (int u = 0; u < U; ++u) {
                nx[u] = IO::raw(x + static_cast<int64_t>(min(t + u, tn)) * a.xt);
                nd[u] = IO::raw(dy + static_cast<int64_t>(min(t + u, tn)) * g.dyt);
            }
        };
        if (t0 <= tn) fetch(t0);
        for (int tb = t0; tb < te; tb += U) {
            typename IO::Raw rx[U], rd[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                rx[u] = tb + u <= tn ? nx[u] : IO::zero();
                rd[u] = tb + u <= tn ? nd[u] : IO::zero();
            }
            if (tb + U <= tn) fetch(tb + U);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = tb + u;
                if (t >= te) break;
                float d[V];
                IO::unpack(rx[u], win[K - 1]);
                IO::unpack(rd[u], d);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (a.silu) {  // d/dz z s = s (1 + z (1 - s))
                        float z = bv[v];
#pragma unroll
                        for (int k = 0; k < K; ++k) z = fmaf(wk[k][v], win[k][v], z);
                        const float s = sigmoid_f(z);
                        d[v] *= s * fmaf(z, 1.0f - s, 1.0f);
                    }
                    if (t >= n) d[v] = 0.f;
                    gw[K - 1][v] = d[v];
                    if (t < t1) {
                        db[v] += d[v];
#pragma unroll
                        for (int k = 0; k < K; ++k) dw[k][v] = fmaf(d[v], win[k][v], dw[k][v]);
                    }
                }
                const int e = t - (K - 1);  // the row whose terms g_e .. g_{e+K-1} are complete
                if (e >= t0 || t0 == 0) {
                    float o[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        o[v] = 0.f;
#pragma unroll
                        for (int k = 0; k < K; ++k) o[v] = fmaf(wk[k][v], gw[K - 1 - k][v], o[v]);
                    }
                    if (dso && e >= n - (K - 1) && e < n) {  // this row is in the state afterwards
                        float q[V];
                        vec_load<T, V>(dso + static_cast<int64_t>(e - n + K - 1) * a.C, q);
#pragma unroll
                        for (int v = 0; v < V; ++v) o[v] += q[v];
                    }
                    if (e >= 0) {
                        IO::store(dx + static_cast<int64_t>(e) * g.dxt, o);
                    } else if (ds) {
                        IO::store(ds + static_cast<int64_t>(e + K - 1) * a.C, o);
                    }
                }
#pragma unroll
                for (int k = 0; k < K - 1; ++k)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        win[k][v] = win[k + 1][v];
                        gw[k][v] = gw[k + 1][v];
                    }
            }
        }
    }
    // the workgroup's sums, one of the K + 1 at a time
    float *part = g.ws + (static_cast<int64_t>(b) * gridDim.x + blockIdx.x) * a.C * (K + 1);
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) red[run][lane * V + v] = k < K ? dw[k][v] : db[v];
        __syncthreads();
        if (threadIdx.x < BC * V) {
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < BR; ++r) s += red[r][threadIdx.x];
            const int cc = blockIdx.y * BC * V + threadIdx.x;
            if (cc < a.C) {
                // dw [C,K] first, then db [C]
                part[k < K ? static_cast<int64_t>(cc) * K + k : static_cast<int64_t>(a.C) * K + cc] = s;
            }
        }
    }
}

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

template <int K, typename T>
hipError_t fwd_kt(const ConvArgs &a, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = a.C % V == 0 && a.xb % V == 0 && a.xt % V == 0 && a.yb % V == 0 && a.yt % V == 0 &&
                     aligned(a.x, 16) && aligned(a.y, 16) && aligned(a.state, 16) && aligned(a.state_out, 16);
    const int cw = vec ? V : 1;
    const int gx = (a.C + NT * cw - 1) / (NT * cw);
    // tokens of a thread: as many as leave about four workgroups for each compute unit, 8 .. 64
    int tokens = 64;
    while (tokens > 8 && static_cast<int64_t>(gx) * ((a.L + tokens - 1) / tokens) * a.B < 1024) tokens /= 2;
    while (a.L / tokens > (1 << 22)) tokens *= 2;  // a grid's threads are counted in 32 bits
    const int gy = a.L > 0 ? (a.L + tokens - 1) / tokens : 1;
    const dim3 grid(gy, gx, a.B);
    if (vec)
        hipLaunchKernelGGL((conv_fwd<K, V, T>), grid, dim3(NT), 0, s, a, tokens);
    else
        hipLaunchKernelGGL((conv_fwd<K, 1, T>), grid, dim3(NT), 0, s, a, tokens);
    return hipGetLastError();
}

template <int K, typename T>
hipError_t step_kt(const ConvArgs &a, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = a.C % V == 0 && a.xb % V == 0 && a.yb % V == 0 && aligned(a.x, 16) &&
                     aligned(a.y, 16) && aligned(a.state_out, 16);
    const int64_t n = static_cast<int64_t>(a.B) * (vec ? a.C / V : a.C);
    const unsigned grid = static_cast<unsigned>((n + NT - 1) / NT);
    if (vec)
        hipLaunchKernelGGL((conv_step<K, V, T>), dim3(grid), dim3(NT), 0, s, a);
    else
        hipLaunchKernelGGL((conv_step<K, 1, T>), dim3(grid), dim3(NT), 0, s, a);
    return hipGetLastError();
}

template <int K, typename T>
hipError_t bwd_kt(const ConvBwdArgs &g, hipStream_t s) {
    const ConvArgs &a = g.f;
    constexpr int V = 4;
    constexpr size_t al = V * sizeof(T);
    const bool vec = a.C % V == 0 && a.xb % V == 0 && a.xt % V == 0 && g.dyb % V == 0 && g.dyt % V == 0 &&
                     g.dxb % V == 0 && g.dxt % V == 0 && aligned(a.x, al) && aligned(g.dy, al) &&
                     aligned(g.dx, al) && aligned(a.state, al) && aligned(g.dstate_out, al) &&
                     aligned(g.dstate, al);
    const int cw = (vec ? V : 1) * BC;
    const int rows = a.B ? static_cast<int>(conv_backward_blocks(a.B, a.L, a.C) / a.B) : 0;
    const dim3 grid(rows, (a.C + cw - 1) / cw, a.B);
    if (a.B) {  // with no sequence the sums below are those of no rows
        if (vec)
            hipLaunchKernelGGL((conv_bwd<K, V, T>), grid, dim3(NT), 0, s, g);
        else
            hipLaunchKernelGGL((conv_bwd<K, 1, T>), grid, dim3(NT), 0, s, g);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t stride = static_cast<int64_t>(a.C) * (K + 1);
    ColumnSums c{g.ws, stride, rows * a.B};
    c.add(0, a.C * K, 1, g.dw);
    c.add(static_cast<int64_t>(a.C) * K, a.C, 1, g.dbias);
    return launch_column_sums(c, s);
}

template <template <int, typename> class F, typename A>
hipError_t by_k(int K, int io, const A &a, hipStream_t s) {
    if (io == 1) return K == 2 ? F<2, bf16_t>::run(a, s) : K == 3 ? F<3, bf16_t>::run(a, s) : F<4, bf16_t>::run(a, s);
    return K == 2 ? F<2, float>::run(a, s) : K == 3 ? F<3, float>::run(a, s) : F<4, float>::run(a, s);
}
template <int K, typename T> struct Fwd { static hipError_t run(const ConvArgs &a, hipStream_t s) { return fwd_kt<K, T>(a, s); } };
template <int K, typename T> struct Step { static hipError_t run(const ConvArgs &a, hipStream_t s) { return step_kt<K, T>(a, s); } };
template <int K, typename T> struct Bwd { static hipError_t run(const ConvBwdArgs &a, hipStream_t s) { return bwd_kt<K, T>(a, s); } };

}  // namespace

hipError_t launch_conv_forward(const ConvArgs &a, hipStream_t stream) { return by_k<Fwd>(a.K, a.io, a, stream); }
hipError_t launch_conv_step(const ConvArgs &a, hipStream_t stream) { return by_k<Step>(a.K, a.io, a, stream); }

// partial rows of dw and db: one for each workgroup's tokens
int64_t conv_backward_blocks(int B, int L, int C) {
    (void)C;
    const int64_t per = BT * BR;
    return B * (L > 0 ? (L + per - 1) / per : 1);
}
hipError_t launch_conv_backward(const ConvBwdArgs &a, hipStream_t stream) {
    return by_k<Bwd>(a.f.K, a.f.io, a, stream);
}

}  // namespace ttt
