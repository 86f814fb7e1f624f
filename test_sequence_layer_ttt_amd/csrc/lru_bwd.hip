// Gradients of the gated linear recurrence (formulas of the forward: lru.hpp).
// With G_t the gradient of h_t and K_t = a_t G_t what flows on to h_{t-1},
//     G_t = dy_t + K_{t+1}  (K behind the last token: dstate_out),
//     l_t = G_t (a_t h_{t-1} + sigma(i_t) x_t s'_t)   the gradient of log a_t,
// s' the derivative of s by log a: -a^2 / s (0 where s is 0) or -a. Then
//     dx = G s sigma(i),  di = G s x sigma(i) (1 - sigma(i)),  dstate = K_1,
//     dr = -rate l sigma(r) (1 - sigma(r)),  drate = -sum l sigma(r)   with a rate,
//     dr = l (1 - a)                                                  without.
#include "block.hpp"
#include "lru.hpp"

namespace ttt {
namespace {

using namespace lru;

constexpr int BT = 64;  // tokens of a tile

template <int V> struct Tile {
    static constexpr int CL = CH / V, TG = NT / CL, U = BT / TG;
};

inline __host__ __device__ int tiles(int L) { return (L + BT - 1) / BT; }

__device__ __forceinline__ int live_tokens(const int *lens, int b, int L) {
    return lens ? max(0, min(lens[b], L)) : L;
}

template <typename T> struct Rows {
    const T *x, *r, *i, *dy;
    __device__ __forceinline__ Rows(const LruBwdArgs &g, int b, int c)
        : x(static_cast<const T *>(g.f.x) + b * g.f.xb + c), r(static_cast<const T *>(g.f.r) + b * g.f.rb + c),
          i(g.f.i ? static_cast<const T *>(g.f.i) + b * g.f.ib + c : nullptr),
          dy(static_cast<const T *>(g.dy) + b * g.dyb + c) {}
};

// Each tile's decay A, its own share H of the state behind it and its own
// share K = sum A_t dy_t of what flows out before it: ws[b][tile][3][D].
template <typename T, int V, bool RATE>
__global__ __launch_bounds__(NT) void lru_bwd_shares(LruBwdArgs g) {
    constexpr int TG = Tile<V>::TG, CL = Tile<V>::CL, U = Tile<V>::U;
    __shared__ float2 sm[TG][CH];
    __shared__ float smk[TG][CH];
    const LruArgs &a = g.f;
    const int lane = threadIdx.x % CL, run = threadIdx.x / CL;
    const int b = blockIdx.z, tile = blockIdx.x, c0 = blockIdx.y * CH, c = c0 + lane * V;
    const int n = live_tokens(a.lens, b, a.L);
    const int t0 = tile * BT + run * U, t1 = min(t0 + U, n);
    float A[V], H[V], K[V], rate[V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = K[v] = 0.f, rate[v] = 0.f;
    if (RATE && c < a.D) load_rate<V>(a.rate + c, rate);
    if (c < a.D && t0 < t1) {
        const Rows<T> p(g, b, c);
        for (int t = t0; t < t1; ++t) {
            float xv[V], rv[V], iv[V] = {}, dv[V];
            vec_load<T, V>(p.x + t * a.xt, xv);
            vec_load<T, V>(p.r + t * a.rt, rv);
            vec_load<T, V>(p.dy + t * g.dyt, dv);
            if (p.i) vec_load<T, V>(p.i + t * a.it, iv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Gate k = gate<RATE>(rv[v], rate[v]);
                float u = k.s * xv[v];
                if (p.i) u *= sigmoid(iv[v]);
                H[v] = fmaf(k.a, H[v], u);
                A[v] *= k.a;
                K[v] = fmaf(A[v], dv[v], K[v]);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sm[run][lane * V + v] = make_float2(A[v], H[v]);
        smk[run][lane * V + v] = K[v];
    }
    __syncthreads();
    const int cc = c0 + threadIdx.x;
    if (threadIdx.x < CH && cc < a.D) {
        float2 all = make_float2(1.f, 0.f);
        float k = 0.f;
#pragma unroll
        for (int q = 0; q < TG; ++q) {
            const float2 s = sm[q][threadIdx.x];
            k = fmaf(all.x, smk[q][threadIdx.x], k);
            all = make_float2(all.x * s.x, fmaf(s.x, all.y, s.y));
        }
        float *w = a.ws + (static_cast<int64_t>(b) * tiles(a.L) + tile) * 3 * a.D + cc;
        w[0] = all.x;
        w[a.D] = all.y;
        w[2 * static_cast<int64_t>(a.D)] = k;
    }
}

// The state before each tile over its H, and what flows into it from behind over its K.
__global__ __launch_bounds__(NT) void lru_bwd_carry(LruBwdArgs g) {
    const LruArgs &a = g.f;
    const int c = blockIdx.x * NT + threadIdx.x, b = blockIdx.y, n = tiles(a.L);
    if (c >= a.D) return;
    const int64_t row = static_cast<int64_t>(b) * a.D + c, D = a.D;
    float *w = a.ws + static_cast<int64_t>(b) * n * 3 * D + c;
    if (blockIdx.z == 0) {
        float h = a.state ? a.state[row] : 0.f;
        for (int k = 0; k < n; ++k, w += 3 * D) {
            const float A = w[0], H = w[D];
            w[D] = h;
            h = fmaf(A, h, H);
        }
    } else {
        float q = g.dstate_out ? g.dstate_out[row] : 0.f;
        w += 3 * D * (n - 1);
        for (int k = 0; k < n; ++k, w -= 3 * D) {
            const float A = w[0], K = w[2 * D];
            w[2 * D] = q;
            q = fmaf(A, q, K);
        }
    }
}

template <typename T, int V, bool RATE>
__global__ __launch_bounds__(NT) void lru_bwd_grads(LruBwdArgs g) {
    typedef VecIO<T, V> IO;
    constexpr int TG = Tile<V>::TG, CL = Tile<V>::CL, U = Tile<V>::U;
    __shared__ float2 sm[TG][CH];
    __shared__ float smk[TG][CH];
    const LruArgs &a = g.f;
    const int lane = threadIdx.x % CL, run = threadIdx.x / CL;
    const int b = blockIdx.z, tile = blockIdx.x, c0 = blockIdx.y * CH, c = c0 + lane * V;
    const int n = live_tokens(a.lens, b, a.L), nt = tiles(a.L);
    const int t0 = tile * BT + run * U;
    const bool in = c < a.D;
    const Rows<T> p(g, b, c);
    float A[V], H[V], K[V], rate[V];
    float xv[U][V], dv[U][V], gi[U][V], ni[U][V];
    Gate k[U][V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = K[v] = 0.f, rate[v] = 0.f;
    if (RATE && in) load_rate<V>(a.rate + c, rate);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int t = t0 + u;
        if (in && t < n) {
            float rv[V], iv[V] = {};
            vec_load<T, V>(p.x + t * a.xt, xv[u]);
            vec_load<T, V>(p.r + t * a.rt, rv);
            vec_load<T, V>(p.dy + t * g.dyt, dv[u]);
            if (p.i) vec_load<T, V>(p.i + t * a.it, iv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                k[u][v] = gate<RATE>(rv[v], rate[v]);
                gi[u][v] = 1.f, ni[u][v] = 0.f;
                if (p.i) gi[u][v] = sigmoid2(iv[v], &ni[u][v]);
            }
        } else {  // leaves the state and the gradients as they are
#pragma unroll
            for (int v = 0; v < V; ++v) {
                k[u][v] = Gate{1.f, 0.f, 0.f, 0.f, 0.f};
                xv[u][v] = dv[u][v] = gi[u][v] = ni[u][v] = 0.f;
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            H[v] = fmaf(k[u][v].a, H[v], k[u][v].s * gi[u][v] * xv[u][v]);
            A[v] *= k[u][v].a;
            K[v] = fmaf(A[v], dv[u][v], K[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        sm[run][lane * V + v] = make_float2(A[v], H[v]);
        smk[run][lane * V + v] = K[v];
    }
    __syncthreads();
    const int64_t D = a.D, row = static_cast<int64_t>(b) * D;
    const int cs = threadIdx.x % CH, cc = c0 + cs;
    const float *w = a.ws + (static_cast<int64_t>(b) * nt + tile) * 3 * D;
    static_assert(NT == 2 * CH, "one half of the threads for each direction");
    if (threadIdx.x < CH) {  // the state before each run over its H
        float h = cc < D ? (nt > 1 ? w[D + cc] : a.state ? a.state[row + cc] : 0.f) : 0.f;
#pragma unroll
        for (int q = 0; q < TG; ++q) {
            const float2 s = sm[q][cs];
            sm[q][cs].y = h;
            h = fmaf(s.x, h, s.y);
        }
    } else {  // and what flows into each run from behind over its K
        float f = cc < D ? (nt > 1 ? w[2 * D + cc] : g.dstate_out ? g.dstate_out[row + cc] : 0.f) : 0.f;
#pragma unroll
        for (int q = TG - 1; q >= 0; --q) {
            const float s = sm[q][cs].x, own = smk[q][cs];
            smk[q][cs] = f;
            f = fmaf(s, f, own);
        }
    }
    __syncthreads();
    float hp[U][V], dr[V] = {};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        H[v] = sm[run][lane * V + v].y;
        K[v] = smk[run][lane * V + v];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            hp[u][v] = H[v];
            H[v] = fmaf(k[u][v].a, H[v], k[u][v].s * gi[u][v] * xv[u][v]);
        }
    }
    T *dx = static_cast<T *>(g.dx) + b * g.dxb + c, *drp = static_cast<T *>(g.dr) + b * g.drb + c;
    T *di = g.di ? static_cast<T *>(g.di) + b * g.dib + c : nullptr;
#pragma unroll
    for (int u = U - 1; u >= 0; --u) {
        const int t = t0 + u;
        float ox[V], orr[V], oi[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Gate q = k[u][v];
            const float G = dv[u][v] + K[v], x = xv[u][v], e = gi[u][v];
            K[v] = q.a * G;
            const float gs = G * q.s;
            ox[v] = gs * e;
            oi[v] = gs * x * e * ni[u][v];
            float l;
            if constexpr (RATE) {
                const float slope = q.s > 0.f ? q.a * q.a * __builtin_amdgcn_rcpf(q.s) : 0.f;
                l = G * fmaf(q.a, hp[u][v], -e * x * slope);
                dr[v] = fmaf(-l, q.g, dr[v]);
                orr[v] = -l * (rate[v] * 0.693147181f) * q.g * q.ng;
            } else {
                l = G * q.a * (hp[u][v] - e * x);
                orr[v] = l * q.o;
            }
        }
        if (in && t < a.L) {
            IO::store(dx + t * g.dxt, ox);
            IO::store(drp + t * g.drt, orr);
            if (di) IO::store(di + t * g.dit, oi);
        }
    }
    if (in && g.dstate && tile == 0 && run == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) g.dstate[row + c + v] = K[v];
    }
    if constexpr (RATE) {  // the tile's sums, in the order of its runs
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) smk[run][lane * V + v] = dr[v];
        __syncthreads();
        if (threadIdx.x < CH && cc < D) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < TG; ++q) s += smk[q][cs];
            float *part = a.ws + (nt > 1 ? static_cast<int64_t>(a.B) * nt * 3 * D : 0);
            part[(static_cast<int64_t>(b) * nt + tile) * D + cc] = s;
        }
    }
}

// L = 0: the state's gradient passes through
__global__ __launch_bounds__(NT) void lru_bwd_pass(LruBwdArgs g) {
    const int64_t k = static_cast<int64_t>(blockIdx.x) * NT + threadIdx.x;
    if (k < static_cast<int64_t>(g.f.B) * g.f.D) g.dstate[k] = g.dstate_out ? g.dstate_out[k] : 0.f;
}

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

template <typename T, int V, bool RATE> hipError_t backward(const LruBwdArgs &g, hipStream_t s) {
    const LruArgs &a = g.f;
    const int nt = tiles(a.L);
    const int64_t rows = static_cast<int64_t>(a.B) * nt;
    if (!nt) {
        const int64_t n = static_cast<int64_t>(a.B) * a.D;
        if (g.dstate && n)
            hipLaunchKernelGGL(lru_bwd_pass, dim3(static_cast<unsigned>((n + NT - 1) / NT)), dim3(NT), 0, s, g);
    } else if (a.B) {
        const dim3 grid(nt, (a.D + CH - 1) / CH, a.B);
        if (nt > 1) {
            hipLaunchKernelGGL((lru_bwd_shares<T, V, RATE>), grid, dim3(NT), 0, s, g);
            hipLaunchKernelGGL(lru_bwd_carry, dim3((a.D + NT - 1) / NT, a.B, 2), dim3(NT), 0, s, g);
        }
        hipLaunchKernelGGL((lru_bwd_grads<T, V, RATE>), grid, dim3(NT), 0, s, g);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !RATE) return e;
    ColumnSums c{a.ws + (nt > 1 ? rows * 3 * a.D : 0), a.D, static_cast<int>(rows)};
    c.add(0, a.D, 1, g.drate);
    return launch_column_sums(c, s);
}

template <typename T> hipError_t backward_t(const LruBwdArgs &g, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const LruArgs &a = g.f;
    const bool vec = a.D % V == 0 && (a.xb | a.xt | a.rb | a.rt | g.dyb | g.dyt | g.dxb | g.dxt | g.drb | g.drt) % V == 0 &&
                     (!a.i || (a.ib | a.it | g.dib | g.dit) % V == 0) && aligned(a.x, 16) && aligned(a.r, 16) &&
                     aligned(a.i, 16) && aligned(g.dy, 16) && aligned(g.dx, 16) && aligned(g.dr, 16) && aligned(g.di, 16);
    if (vec) return a.rate ? backward<T, V, true>(g, s) : backward<T, V, false>(g, s);
    return a.rate ? backward<T, 1, true>(g, s) : backward<T, 1, false>(g, s);
}

}  // namespace

int64_t lru_backward_floats(int B, int L, int D) {
    const int64_t n = tiles(L);
    return (n > 1 ? 4 : 1) * n * B * D;
}
hipError_t launch_lru_backward(const LruBwdArgs &g, hipStream_t s) {
    return g.f.io ? backward_t<bf16_t>(g, s) : backward_t<float>(g, s);
}

}  // namespace ttt
