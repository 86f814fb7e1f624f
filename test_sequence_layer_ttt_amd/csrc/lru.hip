// Gated linear recurrence, a prompt and a single token (formulas: lru.hpp).
#include "lru.hpp"

namespace ttt {
namespace {

using namespace lru;

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

// One pass over the prompt. A workgroup takes a tile of T tokens x 128 channels:
// a thread scans V channels of U consecutive tokens from a zero state, with the
// running state and decay of each in registers; LDS joins the tile's runs, and
// what the tile does to a state, (A, H): h -> A h + H, is published for the
// tiles behind it. With the state before the tile known, a token's output is
// A_t first + H_t.
//
// The state before a tile: tiles are joined in groups of GROUP; a tile takes the
// state behind the group before its own and applies, in their order, the (A, H)
// of the tiles before it in its group; the last tile of a group publishes the
// state behind it. So the order of the sums is fixed, and a prompt of n tiles is a
// chain of n / GROUP links.
//
// Tiles wait for tiles of their own column (a sequence's 128 channels): each takes
// its place by the column's counter as it starts, so that whatever a tile waits
// for has started before it and waits for earlier ones alone. A counter for each
// column, on lines of their own: one for all cost 8 ns a tile, one after the other.
// A published value carries its own flag: a word is ready where it is not all ones
// (cleared to that before; a NaN of this very pattern is published as another NaN).
// Words are written and read as single atomics at the scope of the device, past the
// XCDs' L2 caches.
//
// What bounds it is HBM: every row is read and written once. 2 x 8192 tokens of 2048
// bf16 channels (268 MB) take 57 us, 32768 without input gates (403 MB) 76 us, 4.7 and
// 5.3 TB/s, and lru_clear 5 us before them. Groups of 8 tiles, at 32768 tokens: 83 us a
// call; of 4 95 (a chain of twice as many links), of 16 86 (more shares to join for a tile).
constexpr int GROUP = 8;
constexpr uint32_t WAIT32 = 0xffffffffu;
constexpr uint64_t WAIT64 = 0xffffffffffffffffull;
// About a second. What a tile waits for comes from tiles that are on the chip, microseconds later;
// a word that never comes (a workspace that something else writes) is a NaN then, to the column's end.
constexpr int POLLS = 1 << 20;

struct Plan {
    int tokens;  // of a tile
    int64_t tiles, groups;
};

// workspace: the columns' counters, then the tiles' (A, H) [B][tiles][D], then the states behind groups [B][groups][D]
constexpr int LINE = 16;  // words
struct Words {
    uint32_t *place;
    uint64_t *share;
    uint32_t *state;
    __device__ __forceinline__ Words(float *ws, int64_t columns, int64_t shares)
        : place(reinterpret_cast<uint32_t *>(ws)), share(reinterpret_cast<uint64_t *>(ws + LINE * columns)),
          state(reinterpret_cast<uint32_t *>(ws + LINE * columns + 2 * shares)) {}
};
template <typename W> __device__ __forceinline__ W peek(const W *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W> __device__ __forceinline__ void publish(W *p, W v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W> __device__ __forceinline__ W await(const W *p, W v, W wait) {
    for (int n = 0; v == wait && n < POLLS; ++n) {
        __builtin_amdgcn_s_sleep(2);
        v = peek(p);
    }
    return v;
}

__global__ __launch_bounds__(NT) void lru_clear(uint4 *p, int64_t n) {
    const int64_t k = static_cast<int64_t>(blockIdx.x) * NT + threadIdx.x;
    if (k < n) p[k] = make_uint4(WAIT32, WAIT32, WAIT32, WAIT32);
}

// A run's own scan from a zero state: (A, H) behind each token, all loads asked for at
// once. FULL: a whole tile (8k prompt of 2 x 2048 channels 71 -> 66 us, 32k 91 -> 83).
// Otherwise rows past the sequence's end are read from its last.
template <typename T, int V, int U, bool RATE, bool GATED, bool FULL>
__device__ __forceinline__ void own_scan(const LruArgs &a, int b, int c, int t0, int n, bool some, const float (&rate)[V],
                                         float (&A)[V], float (&H)[V], float (&At)[U][V], float (&Ht)[U][V]) {
    typedef VecIO<T, V> IO;
    const T *x = static_cast<const T *>(a.x) + b * a.xb + c, *r = static_cast<const T *>(a.r) + b * a.rb + c;
    const T *ig = static_cast<const T *>(a.i) + b * a.ib + c;
    typename IO::Raw rx[U], rr[U], ri[U];
    if (FULL || some) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = FULL ? t0 + u : min(t0 + u, n - 1);
            rx[u] = IO::raw(x + t * a.xt);
            rr[u] = IO::raw(r + t * a.rt);
            if (GATED) ri[u] = IO::raw(ig + t * a.it);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (FULL || (some && t0 + u < n)) {
            float xv[V], rv[V], iv[V] = {}, d[V], w[V];
            IO::unpack(rx[u], xv);
            IO::unpack(rr[u], rv);
            if (GATED) IO::unpack(ri[u], iv);
            token<V, RATE>(xv, rv, iv, GATED, rate, d, w);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                H[v] = fmaf(d[v], H[v], w[v]);
                A[v] *= d[v];
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) At[u][v] = A[v], Ht[u][v] = H[v];
        if (FULL) __builtin_amdgcn_sched_barrier(0);
    }
}

template <typename T, int V, int U, bool RATE, bool GATED, bool MANY>
__global__ __launch_bounds__(NT) void lru_scan(LruArgs a, int nch, int ngr) {
    typedef VecIO<T, V> IO;
    constexpr int CL = CH / V, TG = NT / CL;  // lanes along the channels, runs of tokens
    __shared__ float2 sm[TG][CH];
    __shared__ float sfirst[CH];
    __shared__ uint32_t place;
    const int lane = threadIdx.x % CL, run = threadIdx.x / CL;
    // MANY: a grid of columns (the faster) by tiles; else of channels by sequences. Workgroups
    // go to the XCDs round robin: each round starts a column further, so that an XCD does not
    // keep to a few columns, whose lines lie in few of its L2's channels (32k prompt: 102 -> 95 us).
    const int ncb = (a.D + CH - 1) / CH, ncol = ncb * a.B;
    const int column = MANY ? (blockIdx.x + blockIdx.x / ncol) % ncol : 0;
    const int cb = MANY ? column % ncb : blockIdx.x, b = MANY ? column / ncb : blockIdx.y;
    const Words words(a.ws, static_cast<int64_t>(ncb) * a.B, static_cast<int64_t>(a.B) * nch * a.D);
    if (MANY && threadIdx.x == 0) place = atomicAdd(words.place + LINE * column, 1u) + 1;  // from all ones on
    const int c0 = cb * CH, c = c0 + lane * V;
    const int n = live_tokens(a.lens, b, a.L);
    float A[V], H[V], At[U][V], Ht[U][V], rate[V];
    const bool in = c < a.D;
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f, rate[v] = 0.f;
    if (RATE && in) load_rate<V>(a.rate + c, rate);
    if constexpr (MANY) __syncthreads();
    const int k = MANY ? static_cast<int>(min(place, static_cast<uint32_t>(nch - 1))) : 0, t0 = (k * TG + run) * U;
    const bool some = in && t0 < n;
    if (whole(k, TG * U, n, c0, a.D))
        own_scan<T, V, U, RATE, GATED, true>(a, b, c, t0, n, some, rate, A, H, At, Ht);
    else
        own_scan<T, V, U, RATE, GATED, false>(a, b, c, t0, n, some, rate, A, H, At, Ht);
    // the runs before each run, and the tile's own (A, H)
#pragma unroll
    for (int v = 0; v < V; ++v) sm[run][lane * V + v] = make_float2(A[v], H[v]);
    __syncthreads();
    const int64_t row = static_cast<int64_t>(b) * a.D;
    const int cc = c0 + threadIdx.x;
    if (threadIdx.x < CH) {
        float2 all = make_float2(1.f, 0.f);
#pragma unroll
        for (int q = 0; q < TG; ++q) {
            const float2 s = sm[q][threadIdx.x];
            sm[q][threadIdx.x] = all;
            all = make_float2(all.x * s.x, fmaf(s.x, all.y, s.y));
        }
        float h = 0.f;
        if (cc < a.D) {
            // the first tile's share holds the state before it, which no other tile reads
            if (k == 0 && a.state) h = a.state[row + cc];
            if constexpr (MANY) {
                const int j = k / GROUP, before = k % GROUP;  // the group, tiles before this one in it
                const bool ends = before == GROUP - 1;
                uint64_t *share = words.share + (static_cast<int64_t>(b) * nch + k) * a.D + cc;
                uint32_t *state = words.state + (static_cast<int64_t>(b) * ngr + j) * a.D + cc;
                if (!ends && k + 1 < nch) {
                    const float own = k == 0 ? fmaf(all.x, h, all.y) : all.y;
                    uint64_t w = static_cast<uint64_t>(__float_as_uint(own)) << 32 | __float_as_uint(all.x);
                    publish(share, w == WAIT64 ? w << 1 >> 1 : w);
                }
                uint64_t w[GROUP - 1];
#pragma unroll
                for (int q = 0; q < GROUP - 1; ++q)
                    w[q] = q < before ? peek(share - static_cast<int64_t>(before - q) * a.D) : 0;
                if (j > 0) h = __uint_as_float(await(state - a.D, peek(state - a.D), WAIT32));
#pragma unroll
                for (int q = 0; q < GROUP - 1; ++q)
                    if (q < before) {
                        const uint64_t p = await(share - static_cast<int64_t>(before - q) * a.D, w[q], WAIT64);
                        h = fmaf(__uint_as_float(static_cast<uint32_t>(p)), h, __uint_as_float(static_cast<uint32_t>(p >> 32)));
                    }
                if (ends && k + 1 < nch) {
                    const uint32_t s = __float_as_uint(fmaf(all.x, h, all.y));
                    publish(state, s == WAIT32 ? s >> 1 : s);
                }
            }
        }
        sfirst[threadIdx.x] = h;
    }
    __syncthreads();
    if (!in) return;
    float first[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float2 q = sm[run][lane * V + v];
        first[v] = fmaf(q.x, sfirst[lane * V + v], q.y);
    }
    T *y = static_cast<T *>(a.y) + b * a.yb + c;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int t = t0 + u;
        float o[V] = {};
        if (t < n) {
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = fmaf(At[u][v], first[v], Ht[u][v]);
            stream_store<T, V>(y + t * a.yt, o);
        } else if (t < a.L) {
            IO::store(y + t * a.yt, o);
        }
    }
    if (a.state_out && k == nch - 1 && run == TG - 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) a.state_out[row + c + v] = fmaf(At[U - 1][v], first[v], Ht[U - 1][v]);
    }
}

// L = 0: the state passes through
__global__ __launch_bounds__(NT) void lru_pass(LruArgs a) {
    const int64_t k = value_at();
    if (k < static_cast<int64_t>(a.B) * a.D) a.state_out[k] = a.state ? a.state[k] : 0.f;
}

// A single token: a thread V channels. 64 x 2048 channels: 3.4 us, a launch.
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
    if constexpr (RATE) load_rate<V>(a.rate + c, rate);
    token<V, RATE>(xv, rv, iv, a.i != nullptr, rate, d, u);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = fmaf(d[v], h[v], u[v]);
    VecIO<float, V>::store(a.state_out + b * a.D + c, h);
    IO::store(static_cast<T *>(a.y) + b * a.yb + c, h);
}

template <typename T> bool vectors(const LruArgs &a) {
    constexpr int V = 16 / sizeof(T);
    return a.D % V == 0 && (a.xb | a.xt | a.rb | a.rt | a.yb | a.yt) % V == 0 && (!a.i || (a.ib | a.it) % V == 0) &&
           aligned(a.x, 16) && aligned(a.r, 16) && aligned(a.i, 16) && aligned(a.y, 16);
}

// Tiles of `most` tokens, shorter ones where that would leave fewer than four for each
// compute unit.
int tile_tokens(int B, int L, int D, int most) {
    const int64_t wide = (static_cast<int64_t>(D) + CH - 1) / CH * B;
    int tokens = most;
    while (tokens > 32 && wide * ((L + tokens - 1) / tokens) < 1024) tokens /= 2;
    return tokens;
}
Plan plan(int L, int tokens) {
    Plan p{tokens, (static_cast<int64_t>(L) + tokens - 1) / tokens, 0};
    p.groups = p.tiles / GROUP;
    return p;
}
int64_t floats(const Plan &p, int B, int D) {  // in whole 16 bytes
    const int64_t columns = (static_cast<int64_t>(D) + CH - 1) / CH * B;
    return p.tiles > 1 ? (LINE * columns + (2 * p.tiles + p.groups) * B * D + 3) / 4 * 4 : 0;
}

template <typename T, int V, int U, bool RATE, bool GATED> hipError_t scan(const LruArgs &a, const Plan &p, hipStream_t s) {
    const int nch = static_cast<int>(p.tiles), ngr = static_cast<int>(p.groups);
    const int ncb = (a.D + CH - 1) / CH;
    if (nch > 1) {
        const dim3 grid(static_cast<unsigned>(nch) * ncb * a.B);
        const int64_t words = floats(p, a.B, a.D) / 4;
        hipLaunchKernelGGL(lru_clear, dim3(static_cast<unsigned>((words + NT - 1) / NT)), dim3(NT), 0, s,
                           reinterpret_cast<uint4 *>(a.ws), words);
        hipLaunchKernelGGL((lru_scan<T, V, U, RATE, GATED, true>), grid, dim3(NT), 0, s, a, nch, ngr);
    } else {
        hipLaunchKernelGGL((lru_scan<T, V, U, RATE, GATED, false>), dim3(ncb, a.B), dim3(NT), 0, s, a, nch, ngr);
    }
    return hipGetLastError();
}

template <typename T, int V, int U, bool RATE> hipError_t gated(const LruArgs &a, const Plan &p, hipStream_t s) {
    return a.i ? scan<T, V, U, RATE, true>(a, p, s) : scan<T, V, U, RATE, false>(a, p, s);
}

// 128 tokens where a thread takes 8 channels and there are no input gates (2 x 32768 tokens of
// 2048 channels 146 us, with 64 155) or fewer than 32 columns, whose chain a long prompt waits
// for (32768 of 2048 118, 133). Otherwise 64: with input gates, whose tokens are more work (8 x
// 2048 of 2048 67 -> 64 us, 16 x 4096 223 -> 205), and with fewer channels a thread, whose runs
// are as many times longer (2 x 8192 of 2048 in fp32 117 -> 101, 32768 of 2047 in bf16 320 -> 210).
int most_tokens(int B, int D, int V, bool gated) {
    const int64_t wide = (static_cast<int64_t>(D) + CH - 1) / CH * B;
    return V == 8 && !(gated && wide >= 32) ? 128 : 64;
}

template <typename T, int V, bool RATE> hipError_t forward(const LruArgs &a, hipStream_t s) {
    const Plan p = plan(a.L, lru_forward_tokens(a.B, a.L, a.D, V, a.i != nullptr));
    if (!p.tiles) {  // the caller has asked for the state alone
        hipLaunchKernelGGL(lru_pass, values_grid(static_cast<int64_t>(a.B) * a.D), dim3(NT), 0, s, a);
        return hipGetLastError();
    }
    constexpr int TG = NT / (CH / V);
    if constexpr (V == 8) {
        if (p.tokens == 128) return gated<T, V, 128 / TG, RATE>(a, p, s);
    }
    return p.tokens == 64 ? gated<T, V, 64 / TG, RATE>(a, p, s) : gated<T, V, 32 / TG, RATE>(a, p, s);
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

// by the sizes alone: of the tiles that need the most
int64_t lru_forward_floats(int B, int L, int D) { return floats(plan(L, tile_tokens(B, L, D, 64)), B, D); }
int lru_forward_tokens(int B, int L, int D, int V, bool gated) {
    return tile_tokens(B, L, D, most_tokens(B, D, V, gated));
}
hipError_t launch_lru_forward(const LruArgs &a, hipStream_t s) {
    return a.io ? forward_t<bf16_t>(a, s) : forward_t<float>(a, s);
}
hipError_t launch_lru_step(const LruArgs &a, hipStream_t s) {
    return a.io ? step_t<bf16_t>(a, s) : step_t<float>(a, s);
}

}  // namespace ttt
