// Gradients of the gated linear recurrence (formulas of the forward: lru.hpp).
// With G_t the gradient of h_t and K_t = a_t G_t what flows on to h_{t-1},
//     G_t = dy_t + K_{t+1}  (K behind the last token: dstate_out),
//     l_t = G_t (a_t h_{t-1} + sigma(i_t) x_t s'_t)   the gradient of log a_t,
// s' the derivative of s by log a: -a^2 / s (0 where s is 0) or -a. Then
//     dx = G s sigma(i),  di = G s x sigma(i) (1 - sigma(i)),  dstate = K_1,
//     dr = -rate l sigma(r) (1 - sigma(r)),  drate = -sum l sigma(r)   with a rate,
//     dr = l (1 - a)                                                  without.
//
// Two passes over the inputs: lru_bwd_shares gives what each tile does to the state and
// to K, lru_bwd_carry the values at the tiles' borders from those (both directions at
// once), lru_bwd_grads walks again with them. A tile needs both directions, and one pass that
// got both from its neighbours would need all tiles of a column on the chip at once; a
// pass from the last token on could take the states before its tiles from a first one over
// x, r and i alone. Eleven rows are moved
// instead of seven: for 2 x 8192 tokens of 2048 bf16 channels 45 + 8 + 102 us, and 6 for
// drate's sums; the passes run at 5.9 and 4.6 TB/s (a large copy: 5.0). A gate is
// formed again on the way back rather than held: held, a thread takes 182 registers
// instead of 158, and 187 us instead of 178. In fp32 107 + 8 + 189 + 6 us; rows of 2047
// bf16 channels, value by value, 79 + 12 + 181 + 7. 16 x 32768 tokens of 16 channels, where
// drate's 16384 partial rows are one workgroup's, 72 + 13 + 161 + 87.
#include "block.hpp"
#include "lru.hpp"

namespace ttt {
namespace {

using namespace lru;

// A tile's tokens: 32, or 16 where that would leave fewer than four workgroups for each
// compute unit. 64 take more registers than two waves a SIMD have: 2 x 8192 tokens of 2048
// channels 200 us, 178 with 32.
int tile_tokens(int B, int L, int D) {
    const int64_t wide = (static_cast<int64_t>(D) + CH - 1) / CH * B;
    int t = 32;
    while (t > 16 && wide * ((L + t - 1) / t) < 1024) t /= 2;
    return t;
}

// U tokens of V channels as stored, all asked for at once; rows past the
// sequence's end are read from its last.
template <typename T, int V, int U, bool GATED, bool FULL> struct Tokens {
    typename VecIO<T, V>::Raw x[U], r[U], i[U], dy[U];
    __device__ __forceinline__ Tokens(const LruBwdArgs &g, int b, int c, int t0, int n) {
        const LruArgs &a = g.f;
        const T *px = static_cast<const T *>(a.x) + b * a.xb + c, *pr = static_cast<const T *>(a.r) + b * a.rb + c,
                *pd = static_cast<const T *>(g.dy) + b * g.dyb + c, *pi = static_cast<const T *>(a.i) + b * a.ib + c;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = FULL ? t0 + u : min(t0 + u, n - 1);
            x[u] = VecIO<T, V>::raw(px + t * a.xt);
            r[u] = VecIO<T, V>::raw(pr + t * a.rt);
            dy[u] = VecIO<T, V>::raw(pd + t * g.dyt);
            if (GATED) i[u] = VecIO<T, V>::raw(pi + t * a.it);
        }
    }
    Tokens() = default;
};

// Each tile's decay A, its own share H of the state behind it and its own
// share K = sum A_t dy_t of what flows out before it: ws[b][tile][3][D].
template <typename T, int V, int U, bool RATE, bool GATED, bool FULL>
__device__ __forceinline__ void shares(const LruBwdArgs &g, int nt, int n, float2 (*sm)[CH], float (*smk)[CH]) {
    constexpr int CL = CH / V, TG = NT / CL;  // lanes along the channels, runs of tokens
    const LruArgs &a = g.f;
    const int lane = threadIdx.x % CL, run = threadIdx.x / CL;
    const int b = blockIdx.z, tile = blockIdx.x, c0 = blockIdx.y * CH, c = c0 + lane * V;
    const int t0 = (tile * TG + run) * U;
    float A[V], H[V], K[V], rate[V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = K[v] = 0.f, rate[v] = 0.f;
    if (RATE && (FULL || c < a.D)) load_rate<V>(a.rate + c, rate);
    if (FULL || (c < a.D && t0 < n)) {
        const Tokens<T, V, U, GATED, FULL> p(g, b, c, t0, n);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!FULL && t0 + u >= n) continue;
            float xv[V], rv[V], iv[V] = {}, dv[V];
            VecIO<T, V>::unpack(p.x[u], xv);
            VecIO<T, V>::unpack(p.r[u], rv);
            VecIO<T, V>::unpack(p.dy[u], dv);
            if (GATED) VecIO<T, V>::unpack(p.i[u], iv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Gate k = gate<RATE>(rv[v], rate[v]);
                float w = k.s * xv[v];
                if (GATED) w *= sigmoid(iv[v]);
                H[v] = fmaf(k.a, H[v], w);
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
    if (threadIdx.x < CH && (FULL || cc < a.D)) {
        float2 all = make_float2(1.f, 0.f);
        float k = 0.f;
#pragma unroll
        for (int q = 0; q < TG; ++q) {
            const float2 s = sm[q][threadIdx.x];
            k = fmaf(all.x, smk[q][threadIdx.x], k);
            all = make_float2(all.x * s.x, fmaf(s.x, all.y, s.y));
        }
        float *w = a.ws + (static_cast<int64_t>(b) * nt + tile) * 3 * a.D + cc;
        w[0] = all.x;
        w[a.D] = all.y;
        w[2 * static_cast<int64_t>(a.D)] = k;
    }
}
template <typename T, int V, int U, bool RATE, bool GATED>
__global__ __launch_bounds__(NT) void lru_bwd_shares(LruBwdArgs g, int nt) {
    constexpr int TG = NT / (CH / V);
    __shared__ float2 sm[TG][CH];
    __shared__ float smk[TG][CH];
    const int n = live_tokens(g.f.lens, blockIdx.z, g.f.L);
    if (whole(blockIdx.x, TG * U, n, blockIdx.y * CH, g.f.D))
        shares<T, V, U, RATE, GATED, true>(g, nt, n, sm, smk);
    else
        shares<T, V, U, RATE, GATED, false>(g, nt, n, sm, smk);
}

// The state before each tile over its H (z = 0), and what flows into it from
// behind over its K (z = 1, the tiles from the last on). 32 channels by 16 runs of
// tiles: a run's (A, H) from its tiles, the runs before it from LDS, then its tiles
// again.
constexpr int CC = 32, CR = 16;

__global__ __launch_bounds__(CC *CR) void lru_bwd_carry(LruBwdArgs g, int n) {
    __shared__ float2 sm[CR][CC];
    const LruArgs &a = g.f;
    const int lane = threadIdx.x % CC, run = threadIdx.x / CC, b = blockIdx.y;
    const int c = blockIdx.x * CC + lane, per = (n + CR - 1) / CR, k0 = min(run * per, n), k1 = min(k0 + per, n);
    const int64_t D = a.D, row = b * D + c;
    const bool back = blockIdx.z != 0, in = c < D;
    const int64_t step = back ? -3 * D : 3 * D;
    float *w = a.ws + (static_cast<int64_t>(b) * n + (back ? n - 1 - k0 : k0)) * 3 * D + c;
    const int64_t h = back ? 2 * D : D;
    constexpr int AHEAD = 8;
    float2 own = make_float2(1.f, 0.f);
    if (in) {
        for (int k = k0; k < k1; k += AHEAD) {
            float A[AHEAD], H[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const float *p = w + (min(k + u, k1 - 1) - k0) * step;
                A[u] = p[0];
                H[u] = p[h];
            }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (k + u < k1) own = make_float2(own.x * A[u], fmaf(A[u], own.y, H[u]));
        }
    }
    sm[run][lane] = own;
    __syncthreads();
    if (!in) return;
    const float *from = back ? g.dstate_out : a.state;
    float q = from ? from[row] : 0.f;
    for (int i = 0; i < run; ++i) q = fmaf(sm[i][lane].x, q, sm[i][lane].y);
    for (int k = k0; k < k1; k += AHEAD) {
        float A[AHEAD], H[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const float *p = w + (min(k + u, k1 - 1) - k0) * step;
            A[u] = p[0];
            H[u] = p[h];
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (k + u < k1) {
                w[(k + u - k0) * step + h] = q;
                q = fmaf(A[u], q, H[u]);
            }
    }
}

template <typename T, int V, int U, bool RATE, bool GATED, bool FULL>
__device__ __forceinline__ void grads(const LruBwdArgs &g, int nt, int n, float2 (*sm)[CH], float (*smk)[CH]) {
    typedef VecIO<T, V> IO;
    constexpr int CL = CH / V, TG = NT / CL;
    const LruArgs &a = g.f;
    const int lane = threadIdx.x % CL, run = threadIdx.x / CL;
    const int b = blockIdx.z, tile = blockIdx.x, c0 = blockIdx.y * CH, c = c0 + lane * V;
    const int t0 = (tile * TG + run) * U;
    const bool in = FULL || c < a.D;
    // held from here to the way back: the rows as stored, and of each value the decay, the scale
    // and the state before it
    float A[V], H[V], K[V], rate[V], da[U][V], ds[U][V], hp[U][V];
    Tokens<T, V, U, GATED, FULL> p;
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = K[v] = 0.f, rate[v] = 0.f;
    const bool some = FULL || (in && t0 < n);
    if (RATE && in) load_rate<V>(a.rate + c, rate);
    if (some) p = Tokens<T, V, U, GATED, FULL>(g, b, c, t0, n);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int v = 0; v < V; ++v) hp[u][v] = H[v], da[u][v] = 1.f, ds[u][v] = 0.f;
        if (FULL || (some && t0 + u < n)) {
            float xv[V], rv[V], iv[V] = {}, dv[V];
            IO::unpack(p.x[u], xv);
            IO::unpack(p.r[u], rv);
            IO::unpack(p.dy[u], dv);
            if (GATED) IO::unpack(p.i[u], iv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Gate k = gate<RATE>(rv[v], rate[v]);
                da[u][v] = k.a;
                ds[u][v] = k.s;
                float w = k.s * xv[v];
                if (GATED) w *= sigmoid(iv[v]);
                H[v] = fmaf(k.a, H[v], w);
                A[v] *= k.a;
                K[v] = fmaf(A[v], dv[v], K[v]);
            }
        }
        if (FULL) __builtin_amdgcn_sched_barrier(0);
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
    float dr[V] = {};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float first = sm[run][lane * V + v].y;
        float P = 1.f;
        K[v] = smk[run][lane * V + v];
#pragma unroll
        for (int u = 0; u < U; ++u) {  // the state before each token, from the run's own share
            hp[u][v] = fmaf(P, first, hp[u][v]);
            P *= da[u][v];
        }
    }
    T *dx = static_cast<T *>(g.dx) + b * g.dxb + c, *drp = static_cast<T *>(g.dr) + b * g.drb + c;
    T *di = static_cast<T *>(g.di) + b * g.dib + c;
#pragma unroll
    for (int u = U - 1; u >= 0; --u) {
        const int t = t0 + u;
        float ox[V] = {}, orr[V] = {}, oi[V] = {};
        if (FULL || (some && t < n)) {
            float xv[V], rv[V] = {}, iv[V] = {}, dv[V];
            IO::unpack(p.x[u], xv);
            IO::unpack(p.dy[u], dv);
            if (RATE) IO::unpack(p.r[u], rv);
            if (GATED) IO::unpack(p.i[u], iv);
#pragma unroll
            for (int v = 0; v < V; ++v) asm volatile("" : "+v"(rv[v]), "+v"(iv[v]));  // formed again, not held
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float at = da[u][v], st = ds[u][v], G = dv[v] + K[v], gs = G * st;
                K[v] = at * G;
                float x = xv[v];  // sigma(i) x
                ox[v] = gs;
                if (GATED) {
                    float ne;
                    const float e = sigmoid2(iv[v], &ne);
                    x *= e;
                    ox[v] = gs * e;
                    oi[v] = gs * x * ne;
                }
                if constexpr (RATE) {
                    float ng;
                    const float q = sigmoid2(rv[v], &ng);
                    const float slope = st > 0.f ? at * at * __builtin_amdgcn_rcpf(st) : 0.f;
                    const float lg = G * fmaf(at, hp[u][v], -x * slope) * q;
                    dr[v] -= lg;
                    orr[v] = -lg * (rate[v] * 0.693147181f) * ng;
                } else {
                    orr[v] = G * at * (hp[u][v] - x) * st;
                }
            }
        }
        if (FULL || (in && t < a.L)) {
            stream_store<T, V>(dx + t * g.dxt, ox);
            stream_store<T, V>(drp + t * g.drt, orr);
            if (GATED) stream_store<T, V>(di + t * g.dit, oi);
        }
        if (FULL) __builtin_amdgcn_sched_barrier(0);
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
template <typename T, int V, int U, bool RATE, bool GATED>
__global__ __launch_bounds__(NT) void lru_bwd_grads(LruBwdArgs g, int nt) {
    constexpr int TG = NT / (CH / V);
    __shared__ float2 sm[TG][CH];
    __shared__ float smk[TG][CH];
    const int n = live_tokens(g.f.lens, blockIdx.z, g.f.L);
    if (whole(blockIdx.x, TG * U, n, blockIdx.y * CH, g.f.D))
        grads<T, V, U, RATE, GATED, true>(g, nt, n, sm, smk);
    else
        grads<T, V, U, RATE, GATED, false>(g, nt, n, sm, smk);
}

// L = 0: the state's gradient passes through
__global__ __launch_bounds__(NT) void lru_bwd_pass(LruBwdArgs g) {
    const int64_t k = value_at();
    if (k < static_cast<int64_t>(g.f.B) * g.f.D) g.dstate[k] = g.dstate_out ? g.dstate_out[k] : 0.f;
}

template <typename T, int V, int U, bool RATE, bool GATED> void tiled(const LruBwdArgs &g, int nt, hipStream_t s) {
    const LruArgs &a = g.f;
    const dim3 grid(nt, (a.D + CH - 1) / CH, a.B);
    if (nt > 1) {
        hipLaunchKernelGGL((lru_bwd_shares<T, V, U, RATE, GATED>), grid, dim3(NT), 0, s, g, nt);
        hipLaunchKernelGGL(lru_bwd_carry, dim3((a.D + CC - 1) / CC, a.B, 2), dim3(CC * CR), 0, s, g, nt);
    }
    hipLaunchKernelGGL((lru_bwd_grads<T, V, U, RATE, GATED>), grid, dim3(NT), 0, s, g, nt);
}

template <typename T, int V, int U, bool RATE> void gated(const LruBwdArgs &g, int nt, hipStream_t s) {
    g.f.i ? tiled<T, V, U, RATE, true>(g, nt, s) : tiled<T, V, U, RATE, false>(g, nt, s);
}

template <typename T, int V, bool RATE> hipError_t backward(const LruBwdArgs &g, hipStream_t s) {
    constexpr int TG = NT / (CH / V);
    const LruArgs &a = g.f;
    const int tokens = tile_tokens(a.B, a.L, a.D), nt = (a.L + tokens - 1) / tokens;
    const int64_t rows = static_cast<int64_t>(a.B) * nt;
    if (!nt) {
        if (g.dstate && a.B)
            hipLaunchKernelGGL(lru_bwd_pass, values_grid(static_cast<int64_t>(a.B) * a.D), dim3(NT), 0, s, g);
    } else if (a.B) {
        if (tokens == 32)
            gated<T, V, 32 / TG, RATE>(g, nt, s);
        else
            gated<T, V, 16 / TG, RATE>(g, nt, s);
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
    const int t = tile_tokens(B, L, D);
    const int64_t n = (static_cast<int64_t>(L) + t - 1) / t;
    return (n > 1 ? 4 : 1) * n * B * D;
}
hipError_t launch_lru_backward(const LruBwdArgs &g, hipStream_t s) {
    return g.f.io ? backward_t<bf16_t>(g, s) : backward_t<float>(g, s);
}

}  // namespace ttt
