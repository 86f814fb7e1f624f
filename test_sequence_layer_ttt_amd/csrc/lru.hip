// Gated linear recurrence, a prompt and a single token (formulas: lru.hpp).
#include "lru.hpp"

namespace ttt {
namespace {

using namespace lru;

// A thread's share of a tile: V channels of U consecutive tokens.
template <int V> struct Tile {
    static constexpr int CL = CH / V;       // lanes along the channels
    static constexpr int TG = NT / CL;      // runs of tokens
    static constexpr int U = TOKENS / TG;   // tokens of a run
};

__device__ __forceinline__ int live_tokens(const int *lens, int b, int L) {
    return lens ? max(0, min(lens[b], L)) : L;
}

// a and u of one token for V channels
template <int V, bool RATE>
__device__ __forceinline__ void token(const float (&x)[V], const float (&r)[V], const float (&i)[V], bool gated,
                                      const float (&rate)[V], float (&d)[V], float (&u)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Gate k = gate<RATE>(r[v], rate[v]);
        d[v] = k.a;
        u[v] = k.s * x[v];
        if (gated) u[v] *= sigmoid(i[v]);
    }
}

// Scan over the runs of a tile: on entry a thread's (A, H) of its run, on exit
// those of all runs before it; the tile's own are returned for channel
// threadIdx.x (threads below CH).
template <int V>
__device__ __forceinline__ float2 tile_scan(float (&A)[V], float (&H)[V], float2 (*sm)[CH]) {
    constexpr int TG = Tile<V>::TG, CL = Tile<V>::CL;
    const int lane = threadIdx.x % CL, run = threadIdx.x / CL;
#pragma unroll
    for (int v = 0; v < V; ++v) sm[run][lane * V + v] = make_float2(A[v], H[v]);
    __syncthreads();
    float2 all = make_float2(1.f, 0.f);
    if (threadIdx.x < CH) {
#pragma unroll
        for (int g = 0; g < TG; ++g) {
            const float2 q = sm[g][threadIdx.x];
            sm[g][threadIdx.x] = all;
            all = make_float2(all.x * q.x, fmaf(q.x, all.y, q.y));
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float2 q = sm[run][lane * V + v];
        A[v] = q.x;
        H[v] = q.y;
    }
    return all;
}

// Each tile's decay and own share of the state behind it: ws[b][chunk][2][D].
template <typename T, int V, bool RATE>
__global__ __launch_bounds__(NT) void lru_shares(LruArgs a) {
    constexpr int TG = Tile<V>::TG, CL = Tile<V>::CL, U = Tile<V>::U;
    __shared__ float2 sm[TG][CH];
    const int lane = threadIdx.x % CL, run = threadIdx.x / CL;
    const int b = blockIdx.z, chunk = blockIdx.x, c0 = blockIdx.y * CH, c = c0 + lane * V;
    const int n = live_tokens(a.lens, b, a.L);
    const int t0 = chunk * TOKENS + run * U, t1 = min(t0 + U, n);
    float A[V], H[V], rate[V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f, rate[v] = RATE && c < a.D ? a.rate[c + v] : 0.f;
    if (c < a.D && t0 < t1) {
        const T *x = static_cast<const T *>(a.x) + b * a.xb + c, *r = static_cast<const T *>(a.r) + b * a.rb + c;
        const T *ig = a.i ? static_cast<const T *>(a.i) + b * a.ib + c : nullptr;
        for (int t = t0; t < t1; ++t) {
            float xv[V], rv[V], iv[V] = {}, d[V], u[V];
            vec_load<T, V>(x + t * a.xt, xv);
            vec_load<T, V>(r + t * a.rt, rv);
            if (ig) vec_load<T, V>(ig + t * a.it, iv);
            token<V, RATE>(xv, rv, iv, ig != nullptr, rate, d, u);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                H[v] = fmaf(d[v], H[v], u[v]);
                A[v] *= d[v];
            }
        }
    }
    const float2 all = tile_scan<V>(A, H, sm);
    const int cc = c0 + threadIdx.x;
    if (threadIdx.x < CH && cc < a.D) {
        float *w = a.ws + (static_cast<int64_t>(b) * chunks(a.L) + chunk) * 2 * a.D;
        w[cc] = all.x;
        w[a.D + cc] = all.y;
    }
}

// The state before each tile, over its share in ws.
__global__ __launch_bounds__(NT) void lru_carry(LruArgs a) {
    const int c = blockIdx.x * NT + threadIdx.x, b = blockIdx.y, n = chunks(a.L);
    if (c >= a.D) return;
    float *w = a.ws + static_cast<int64_t>(b) * n * 2 * a.D + c;
    float h = a.state ? a.state[static_cast<int64_t>(b) * a.D + c] : 0.f;
    for (int k = 0; k < n; ++k, w += 2 * static_cast<int64_t>(a.D)) {
        const float A = w[0], H = w[a.D];
        w[0] = h;
        h = fmaf(A, h, H);
    }
}

template <typename T, int V, bool RATE>
__global__ __launch_bounds__(NT) void lru_outputs(LruArgs a) {
    typedef VecIO<T, V> IO;
    constexpr int TG = Tile<V>::TG, CL = Tile<V>::CL, U = Tile<V>::U;
    __shared__ float2 sm[TG][CH];
    const int lane = threadIdx.x % CL, run = threadIdx.x / CL;
    const int b = blockIdx.z, chunk = blockIdx.x, c0 = blockIdx.y * CH, c = c0 + lane * V;
    const int n = live_tokens(a.lens, b, a.L), nch = chunks(a.L);
    const int t0 = chunk * TOKENS + run * U;
    float A[V], H[V], At[U][V], Ht[U][V], rate[V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f, rate[v] = RATE && c < a.D ? a.rate[c + v] : 0.f;
    const bool in = c < a.D;
    const T *x = static_cast<const T *>(a.x) + b * a.xb + c, *r = static_cast<const T *>(a.r) + b * a.rb + c;
    const T *ig = a.i ? static_cast<const T *>(a.i) + b * a.ib + c : nullptr;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int t = t0 + u;
        if (in && t < n) {
            float xv[V], rv[V], iv[V] = {}, d[V], w[V];
            vec_load<T, V>(x + t * a.xt, xv);
            vec_load<T, V>(r + t * a.rt, rv);
            if (ig) vec_load<T, V>(ig + t * a.it, iv);
            token<V, RATE>(xv, rv, iv, ig != nullptr, rate, d, w);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                H[v] = fmaf(d[v], H[v], w[v]);
                A[v] *= d[v];
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) At[u][v] = A[v], Ht[u][v] = H[v];
    }
    const int64_t row = static_cast<int64_t>(b) * a.D;
    float first[V];
    const float *from = nch > 1 ? a.ws + (static_cast<int64_t>(b) * nch + chunk) * 2 * a.D : a.state ? a.state + row : nullptr;
#pragma unroll
    for (int v = 0; v < V; ++v) first[v] = in && from ? from[c + v] : 0.f;
    tile_scan<V>(A, H, sm);
    if (!in) return;
#pragma unroll
    for (int v = 0; v < V; ++v) first[v] = fmaf(A[v], first[v], H[v]);
    T *y = static_cast<T *>(a.y) + b * a.yb + c;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int t = t0 + u;
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = t < n ? fmaf(At[u][v], first[v], Ht[u][v]) : 0.f;
        if (t < a.L) IO::store(y + t * a.yt, o);
    }
    if (a.state_out && chunk == nch - 1 && run == TG - 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) a.state_out[row + c + v] = fmaf(At[U - 1][v], first[v], Ht[U - 1][v]);
    }
}

// L = 0: the state passes through
__global__ __launch_bounds__(NT) void lru_pass(LruArgs a) {
    const int64_t k = static_cast<int64_t>(blockIdx.x) * NT + threadIdx.x;
    if (k < static_cast<int64_t>(a.B) * a.D) a.state_out[k] = a.state ? a.state[k] : 0.f;
}

template <typename T, int V, bool RATE>
__global__ __launch_bounds__(NT) void lru_step(LruArgs a) {
    typedef VecIO<T, V> IO;
    const int vecs = a.D / V;
    const int64_t k = static_cast<int64_t>(blockIdx.x) * NT + threadIdx.x;
    if (k >= static_cast<int64_t>(a.B) * vecs) return;
    const int64_t b = k / vecs;
    const int c = static_cast<int>(k % vecs) * V;
    float xv[V], rv[V], iv[V] = {}, h[V], d[V], u[V], rate[V] = {};
    vec_load<T, V>(static_cast<const T *>(a.x) + b * a.xb + c, xv);
    vec_load<T, V>(static_cast<const T *>(a.r) + b * a.rb + c, rv);
    if (a.i) vec_load<T, V>(static_cast<const T *>(a.i) + b * a.ib + c, iv);
    vec_load<float, V>(a.state_out + b * a.D + c, h);
    if constexpr (RATE) vec_load<float, V>(a.rate + c, rate);
    token<V, RATE>(xv, rv, iv, a.i != nullptr, rate, d, u);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = fmaf(d[v], h[v], u[v]);
    VecIO<float, V>::store(a.state_out + b * a.D + c, h);
    IO::store(static_cast<T *>(a.y) + b * a.yb + c, h);
}

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

template <typename T> bool vectors(const LruArgs &a) {
    constexpr int V = 16 / sizeof(T);
    return a.D % V == 0 && (a.xb | a.xt | a.rb | a.rt | a.yb | a.yt) % V == 0 && (!a.i || (a.ib | a.it) % V == 0) &&
           aligned(a.x, 16) && aligned(a.r, 16) && aligned(a.i, 16) && aligned(a.y, 16);
}

template <typename T, int V, bool RATE> hipError_t forward(const LruArgs &a, hipStream_t s) {
    const int nch = chunks(a.L);
    if (!nch) {  // the caller has asked for the state alone
        const int64_t n = static_cast<int64_t>(a.B) * a.D;
        hipLaunchKernelGGL(lru_pass, dim3(static_cast<unsigned>((n + NT - 1) / NT)), dim3(NT), 0, s, a);
        return hipGetLastError();
    }
    const dim3 grid(nch, (a.D + CH - 1) / CH, a.B);
    if (nch > 1) {
        hipLaunchKernelGGL((lru_shares<T, V, RATE>), grid, dim3(NT), 0, s, a);
        hipLaunchKernelGGL(lru_carry, dim3((a.D + NT - 1) / NT, a.B), dim3(NT), 0, s, a);
    }
    hipLaunchKernelGGL((lru_outputs<T, V, RATE>), grid, dim3(NT), 0, s, a);
    return hipGetLastError();
}

template <typename T, int V, bool RATE> hipError_t step(const LruArgs &a, hipStream_t s) {
    const int64_t n = static_cast<int64_t>(a.B) * (a.D / V);
    hipLaunchKernelGGL((lru_step<T, V, RATE>), dim3(static_cast<unsigned>((n + NT - 1) / NT)), dim3(NT), 0, s, a);
    return hipGetLastError();
}

template <typename T> hipError_t forward_t(const LruArgs &a, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (vectors<T>(a)) return a.rate ? forward<T, V, true>(a, s) : forward<T, V, false>(a, s);
    return a.rate ? forward<T, 1, true>(a, s) : forward<T, 1, false>(a, s);
}
template <typename T> hipError_t step_t(const LruArgs &a, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    if (vectors<T>(a) && aligned(a.state_out, 16) && aligned(a.rate, 16))
        return a.rate ? step<T, V, true>(a, s) : step<T, V, false>(a, s);
    return a.rate ? step<T, 1, true>(a, s) : step<T, 1, false>(a, s);
}

}  // namespace

int64_t lru_forward_floats(int B, int L, int D) {
    const int64_t n = lru::chunks(L);
    return n > 1 ? 2 * n * B * D : 0;
}
hipError_t launch_lru_forward(const LruArgs &a, hipStream_t s) {
    return a.io ? forward_t<bf16_t>(a, s) : forward_t<float>(a, s);
}
hipError_t launch_lru_step(const LruArgs &a, hipStream_t s) {
    return a.io ? step_t<bf16_t>(a, s) : step_t<float>(a, s);
}

}  // namespace ttt
