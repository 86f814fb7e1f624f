// 8-bit integer product with a scale for each token and each feature,
//     y[m][n] = xs[m] ws[n] sum_k x[m][k] w[n][k] (+ bias[n]),
// the sum exact in 32 bits (K <= 65536: below 2^30), then two products and a
// sum in fp32 and one rounding to y's type. Computed transposed, w as the A
// operand of the 16x16x64 MFMA, so that a lane's four accumulators are four
// consecutive features of one token.
#include "i8_scale.hpp"
#include "vec.hpp"

namespace ttt {
namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;

__device__ __forceinline__ i32x4 mfma_i8(i32x4 a, i32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// Bytes k .. k + 15 of a row of K at any address, zeros from K on: the aligned
// words that hold one of them, shifted together. Every word that is read holds
// a byte of the row.
typedef __attribute__((ext_vector_type(4), aligned(4))) uint32_t word4;

__device__ __forceinline__ i32x4 load16(const int8_t *row, int k, int K) {
    uint32_t d[5] = {};
    const uintptr_t p = reinterpret_cast<uintptr_t>(row + k);
    const uint32_t *q = reinterpret_cast<const uint32_t *>(p & ~static_cast<uintptr_t>(3));
    const uint32_t sh = static_cast<uint32_t>(p & 3);
    if (k + 20 <= K) {  // all five words
        const word4 v = *reinterpret_cast<const word4 *>(q);
        d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
        d[4] = q[4];
    } else if (k < K) {
        const uintptr_t end = reinterpret_cast<uintptr_t>(row + K);
#pragma unroll
        for (int j = 0; j < 5; ++j)
            if (reinterpret_cast<uintptr_t>(q + j) < end) d[j] = q[j];
    }
    const int live = K - k;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t v = __builtin_amdgcn_alignbyte(d[j + 1], d[j], sh);
        const int n = live - 4 * j;
        d[j] = n >= 4 ? v : n <= 0 ? 0u : v & ((1u << (8 * n)) - 1);
    }
    return i32x4{static_cast<int>(d[0]), static_cast<int>(d[1]), static_cast<int>(d[2]), static_cast<int>(d[3])};
}

// E features' scales and biases, asked for before they are needed (without a
// branch, which would wait for them).
template <int E> struct Features {
    float ws[E], bias[E];
    __device__ __forceinline__ Features(const I8Args &a, int n) {
        const float *b = a.bias ? a.bias : a.ws;
        const float with = a.bias ? 1.f : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int f = min(n + e, a.N - 1);
            ws[e] = a.ws[f];
            bias[e] = b[f];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) bias[e] = with != 0.f ? bias[e] : 0.f;
    }
};

// feature n of token m as one of the layer's views
__device__ __forceinline__ uint16_t *view_at(const I8Args &a, int m, int n) {
    const int HD = a.H * 64, v = n / HD, hj = n - v * HD, b = m / a.L, t = m - b * a.L;
    uint16_t *y = static_cast<uint16_t *>(v == 0 ? a.v[0] : v == 1 ? a.v[1] : a.v[2]);
    return y + ((static_cast<int64_t>(b) * a.H + hj / 64) * a.L + t) * 64 + hj % 64;
}

__device__ __forceinline__ void store1(const I8Args &a, int m, int n, float o) {
    if (!a.out_io)
        static_cast<float *>(a.y)[m * a.yr + n] = o;
    else
        *(a.H ? view_at(a, m, n) : static_cast<uint16_t *>(a.y) + (m * a.yr + n)) = f32_to_bf16(o);
}

// features n .. n + 3 of token m, whose scale is sx
__device__ __forceinline__ void store4(const I8Args &a, int m, int n, float sx, const Features<4> &f, i32x4 acc) {
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = fmaf(static_cast<float>(acc[e]) * sx, f.ws[e], f.bias[e]);
    const bool vec = a.vec && n + 4 <= a.N;
    if (a.out_io) {
        // N is a multiple of 64 there: four features of one head
        uint16_t *y = a.H ? view_at(a, m, n) : static_cast<uint16_t *>(a.y) + (m * a.yr + n);
        if (vec) {
            *reinterpret_cast<uint2 *>(y) = make_uint2(tile::pack2(o[0], o[1]), tile::pack2(o[2], o[3]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < a.N) y[e] = f32_to_bf16(o[e]);
        }
    } else {
        float *y = static_cast<float *>(a.y) + (m * a.yr + n);
        if (vec) {
            *reinterpret_cast<float4 *>(y) = make_float4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < a.N) y[e] = o[e];
        }
    }
}

// Any sizes, strides and addresses: a workgroup takes 64 features x 64 tokens,
// a wave 32 x 32 of them, contraction steps of 256 bytes through LDS, the next
// step's rows on their way in registers (bound by their latency: steps of 64 bytes
// took 25.8 us where these take 15, 1551 x 771 x 1037). Rows of 272 bytes: the rows
// of a fragment read lie in distinct banks.
constexpr int GT = 64, GK = 256, GS = GK + 16;

__global__ __launch_bounds__(256) void i8_any(I8Args a) {
    __shared__ __attribute__((aligned(16))) int8_t sw[GT * GS], sx[GT * GS];
    const int nf = (a.N + GT - 1) / GT;
    const int n0 = static_cast<int>(blockIdx.x % nf) * GT, m0 = static_cast<int>(blockIdx.x / nf) * GT;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, c = lane & 15;
    const int row = tid >> 4, part = (tid & 15) * 16;  // rows row, row + 16, ..
    const int8_t *pw[4], *px[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // rows behind the last are read from it; their outputs are not stored
        pw[i] = a.w + static_cast<int64_t>(min(n0 + row + 16 * i, a.N - 1)) * a.wr;
        px[i] = a.x + static_cast<int64_t>(min(m0 + row + 16 * i, a.M - 1)) * a.xr;
    }
    const int wf = (w & 1) * 32, wt = (w >> 1) * 32;
    i32x4 acc[2][2] = {}, nw[4], nx[4];
    auto fetch = [&](int k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            nw[i] = load16(pw[i], k + part, a.K);
            nx[i] = load16(px[i], k + part, a.K);
        }
    };
    fetch(0);
    for (int k = 0; k < a.K; k += GK) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            *reinterpret_cast<i32x4 *>(&sw[(row + 16 * i) * GS + part]) = nw[i];
            *reinterpret_cast<i32x4 *>(&sx[(row + 16 * i) * GS + part]) = nx[i];
        }
        __syncthreads();
        fetch(k + GK);
#pragma unroll
        for (int kk = 0; kk < GK / 64; ++kk) {
            i32x4 fw[2], fx[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fw[i] = *reinterpret_cast<const i32x4 *>(&sw[(wf + 16 * i + c) * GS + 64 * kk + 16 * g]);
                fx[i] = *reinterpret_cast<const i32x4 *>(&sx[(wt + 16 * i + c) * GS + 64 * kk + 16 * g]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = mfma_i8(fx[j], fw[i], acc[i][j]);
        }
        __syncthreads();
    }
    // x as the A operand here: a lane has four tokens of one feature, so that stores of single
    // elements lie 16 together
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int n = n0 + wf + 16 * i + c;
        const Features<1> f(a, n);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float sx[4];
            const int m = m0 + wt + 16 * j + 4 * g;
#pragma unroll
            for (int e = 0; e < 4; ++e) sx[e] = a.xs[min(m + e, a.M - 1)];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (m + e < a.M && n < a.N) store1(a, m + e, n, fmaf(static_cast<float>(acc[i][j][e]) * sx[e], f.ws[0], f.bias[0]));
        }
    }
}

// Few tokens (M <= 16 MT): bound by reading w, and by latency. A workgroup takes
// 16 features and all tokens; its 8 waves split K, each reads its part of w
// straight into the MFMA's layout (lane (g, c): bytes 16 g .. of row c), and LDS
// joins their sums. All of a wave's loads are asked for before the first product
// (up to AHEAD contraction steps).
constexpr int FW = 8, AHEAD = 4;

// 16 bytes of a row from k on, zeros past K; whole chunks at 16-byte addresses or any
template <bool CHUNKS> __device__ __forceinline__ i32x4 row16(const int8_t *row, int k, int K) {
    if constexpr (CHUNKS)
        return k < K ? *reinterpret_cast<const i32x4 *>(row + k) : i32x4{0, 0, 0, 0};
    else
        return load16(row, k, K);
}

// The waves' sums of NT tiles; wave w < NT gets tile w's.
template <int NT> __device__ __forceinline__ i32x4 join(const i32x4 (&acc)[NT], i32x4 (*red)[NT][64]) {
    static_assert(NT <= FW, "a tile for each wave at most");
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int t = 0; t < NT; ++t) red[w][t][lane] = acc[t];
    __syncthreads();
    i32x4 s = {};
    if (w < NT) {
#pragma unroll
        for (int i = 0; i < FW; ++i) s += red[i][w][lane];
    }
    return s;
}

// FT x MT tiles of 16 features x 16 tokens
template <int FT, int MT, bool CHUNKS> __global__ __launch_bounds__(64 * FW) void i8_few(I8Args a) {
    __shared__ i32x4 red[FW][FT * MT][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
    const int n0 = blockIdx.x * 16 * FT;
    const int steps = (a.K + 63) / 64, per = (steps + FW - 1) / FW;
    const int s0 = w * per, s1 = min(s0 + per, steps);
    const int8_t *pw[FT], *px[MT];
#pragma unroll
    for (int f = 0; f < FT; ++f) pw[f] = a.w + static_cast<int64_t>(min(n0 + 16 * f + c, a.N - 1)) * a.wr;
#pragma unroll
    for (int t = 0; t < MT; ++t) px[t] = a.x + static_cast<int64_t>(min(16 * t + c, a.M - 1)) * a.xr;
    const int n = n0 + 16 * (w / MT) + 4 * g, m = 16 * (w % MT) + c;  // the wave's outputs, w < FT MT
    const Features<4> four(a, n);
    const float sx = a.xs[min(m, a.M - 1)];
    i32x4 acc[FT * MT] = {};
    for (int s = s0; s < s1; s += AHEAD) {
        i32x4 fw[AHEAD][FT], fx[AHEAD][MT];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int k = s + i < s1 ? (s + i) * 64 + 16 * g : a.K;
#pragma unroll
            for (int f = 0; f < FT; ++f) fw[i][f] = row16<CHUNKS>(pw[f], k, a.K);
#pragma unroll
            for (int t = 0; t < MT; ++t) fx[i][t] = row16<CHUNKS>(px[t], k, a.K);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int f = 0; f < FT; ++f)
#pragma unroll
                for (int t = 0; t < MT; ++t) acc[f * MT + t] = mfma_i8(fw[i][f], fx[i][t], acc[f * MT + t]);
    }
    const i32x4 sum = join<FT * MT>(acc, red);
    if (w < FT * MT && m < a.M && n < a.N) store4(a, m, n, sx, four, sum);
}

// The same from features, for M <= 16: every workgroup quantises all rows into its
// LDS (rows of `stride` bytes), W threads a row; that is M K values read from the
// chip's caches and one launch less. Its first loads of w are under way meanwhile.
template <typename T, int V, bool CHUNKS>
__global__ __launch_bounds__(64 * FW) void i8_few_features(I8Args a, const T *x, int64_t xr, int W, int stride) {
    extern __shared__ __attribute__((aligned(16))) int8_t sq[];
    __shared__ i32x4 red[FW][1][64];
    __shared__ uint32_t most[16];
    __shared__ float scale[16];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
    const int n0 = blockIdx.x * 16;
    const int steps = (a.K + 63) / 64, per = (steps + FW - 1) / FW;
    const int s0 = w * per, s1 = min(s0 + per, steps);
    const int8_t *pw = a.w + static_cast<int64_t>(min(n0 + c, a.N - 1)) * a.wr;
    i32x4 fw[AHEAD];
    auto ask = [&](int s) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) fw[i] = row16<CHUNKS>(pw, s + i < s1 ? (s + i) * 64 + 16 * g : a.K, a.K);
    };
    ask(s0);
    const int n = n0 + 4 * g;
    const Features<4> four(a, n);
    if (threadIdx.x < 16) most[threadIdx.x] = 0;
    __syncthreads();
    const int at = threadIdx.x % W, first = threadIdx.x / W, rows = 64 * FW / W;
    for (int m = first; m < a.M; m += rows) {  // the bits of the row's largest |x|
        uint32_t mine = 0;
        for (int k = at * V; k < a.K; k += W * V) {
            float v[V];
            vec_load<T, V>(x + m * xr + k, v);
#pragma unroll
            for (int e = 0; e < V; ++e) mine = max(mine, __float_as_uint(v[e]) & 0x7fffffffu);
        }
        atomicMax(&most[m], mine);
    }
    __syncthreads();
    for (int m = first; m < a.M; m += rows) {
        const Scale s(most[m]);
        if (at == 0) scale[m] = s.s;
        for (int k = at * V; k < a.K; k += W * V) {
            float v[V];
            vec_load<T, V>(x + m * xr + k, v);
            s.put<V>(v, sq + m * stride + k);
        }
    }
    __syncthreads();
    const int8_t *px = sq + min(c, a.M - 1) * stride + 16 * g;  // past K: w's zeros
    i32x4 acc[1] = {};
    for (int s = s0; s < s1; s += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (s + i < s1) acc[0] = mfma_i8(fw[i], *reinterpret_cast<const i32x4 *>(px + (s + i) * 64), acc[0]);
        if (s + AHEAD < s1) ask(s + AHEAD);
    }
    const i32x4 sum = join<1>(acc, red);
    if (w == 0 && c < a.M && n < a.N) store4(a, c, n, scale[c], four, sum);
}

// Where logical chunk j of row r of a half lies among its eight: j ^ key(r).
__device__ __forceinline__ int keyA(int r) { return (r & 3) | ((r >> 1) & 4); }

// Workgroup id -> tile. Workgroups go to the 8 XCDs round robin; each XCD takes
// a run of tiles, by fours of feature blocks over all token blocks, so that the
// 32 tiles it works on at a time share 4 blocks of w and 8 of x in its L2.
__device__ __forceinline__ void tile_of(int id, int nfb, int ntb, int *fb, int *tb) {
    const int T = nfb * ntb, q = T / 8, r = T % 8, x = id % 8;
    const int i = x * q + min(x, r) + id / 8;
    const int f0 = i / (4 * ntb) * 4, k = i - f0 * ntb, n = min(4, nfb - f0);
    *fb = f0 + k % n;
    *tb = k / n;
}

struct Lanes {
    Features<8> h[2];
    __device__ __forceinline__ Lanes(const I8Args &a, int n) : h{{a, n}, {a, n + 32}} {}
};

// A lane's 16 features of token m, n .. n + 7 and n + 32 .. n + 39: four accumulators acc(0 .. 3).
template <typename F> __device__ __forceinline__ void store16(const I8Args &a, int m, int n, float sx, const Lanes &f, F acc) {
    if (m >= a.M || n >= a.N) return;
    const bool vec = a.vec && n + 40 <= a.N;
    float o[16];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const i32x4 v = acc(t);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[4 * t + e] = fmaf(static_cast<float>(v[e]) * sx, f.h[t / 2].ws[4 * (t % 2) + e], f.h[t / 2].bias[4 * (t % 2) + e]);
    }
    if (a.out_io) {
        // N is a multiple of 64 there: all of one head
        uint16_t *y = a.H ? view_at(a, m, n) : static_cast<uint16_t *>(a.y) + (m * a.yr + n);
        if (vec) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<uint4 *>(y + 32 * h) =
                    make_uint4(tile::pack2(o[8 * h], o[8 * h + 1]), tile::pack2(o[8 * h + 2], o[8 * h + 3]),
                               tile::pack2(o[8 * h + 4], o[8 * h + 5]), tile::pack2(o[8 * h + 6], o[8 * h + 7]));
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (n + 32 * (e / 8) + e % 8 < a.N) y[32 * (e / 8) + e % 8] = f32_to_bf16(o[e]);
        }
    } else {
        float *y = static_cast<float *>(a.y) + (m * a.yr + n);
        if (vec) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                *reinterpret_cast<float4 *>(y + 32 * (t / 2) + 4 * (t % 2)) = make_float4(o[4 * t], o[4 * t + 1], o[4 * t + 2], o[4 * t + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (n + 32 * (e / 8) + e % 8 < a.N) y[32 * (e / 8) + e % 8] = o[e];
        }
    }
}

// Large products: a workgroup of 8 waves takes 256 features x 256 tokens.
// Contraction steps of 128 bytes; both operands lie in LDS in halves of 128
// rows, two stages of 64 KB, filled by direct global-to-LDS loads.
//  * a wave (wr, wc) takes 64 x 32 of each of the four quadrants (a half of the
//    features by a half of the tokens): 4 x 2 MFMA tiles, and walks them as
//    (0,0), (1,0), (1,1), (0,1), so that a step reads every fragment once;
//  * a quadrant is two sections: M reads the fragments that it or the next
//    quadrant lacks (8 or 4 of 1 KB) and asks for the half of two steps ahead
//    whose place was read last, C is its 16 products. A barrier ends each
//    section, and the waves 4 .. 7 run one section behind the waves 0 .. 3: on
//    each SIMD one wave multiplies while the other one reads;
//  * a half is asked for 7 M sections before it is read: s_waitcnt vmcnt(12) at
//    the end of M leaves the 12 younger loads in flight. That wait and the one
//    for the section's own LDS reads stand before the section's barrier, so
//    behind it every wave's loads have landed, and the place of what was read
//    may be filled again;
//  * rows of 128 bytes, 16-byte chunk j of row r at j ^ key(r): 8 distinct
//    places for the 8 rows that a fragment read touches at once. A's MFMA row
//    4 g + e of tile t is feature 32 (t / 2) + 8 g + 4 (t % 2) + e, so that a lane
//    ends up with twice 8 consecutive features of a token (16 bytes of bf16) and a
//    store of four lanes with 64 bytes;
//  * past K the chunks are read again from the last one and A's are taken as
//    zeros; rows past the end are read from the last one and not stored.
constexpr int BT = 256, BK = 128;

typedef __attribute__((address_space(3))) void lds_void;

// Rows from p on, for loads by a 32-bit offset; the offsets stay within the rows.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const int8_t *p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(p), 0, 0xffffffff, 0x00027000);
}
__device__ __forceinline__ void fence() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void section_end() {  // barrier alone: no wait
    fence();
    __builtin_amdgcn_s_barrier();
    fence();
}

template <bool TAIL> __global__ __launch_bounds__(512, 2) void i8_big(I8Args a, int nfb, int ntb) {
    // halves of A, then of B, each for both stages: 64 KB that one address reaches
    __shared__ __attribute__((aligned(16))) int8_t sm[2][2][2][128 * BK];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, c = lane & 15;
    const int wr = w >> 2, wc = w & 3;
    int fb, tb;
    tile_of(blockIdx.x, nfb, ntb, &fb, &tb);
    const int n0 = fb * BT, m0 = tb * BT;
    const int nk = (a.K + BK - 1) / BK, tail = TAIL ? a.K % BK : 0;  // a multiple of 16

    // loads: a wave's instruction q fills rows 16 w + 8 q .. + 7 of a half
    const auto baseA = buffer(a.w + static_cast<int64_t>(n0) * a.wr), baseB = buffer(a.x + static_cast<int64_t>(m0) * a.xr);
    uint32_t off[4][2];  // of A0, A1, B0, B1 from their base
    const int rl = lane >> 3, pc = lane & 7;
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int r = 16 * w + 8 * q + rl;
            const int ch = pc ^ (h < 2 ? keyA(r) : r & 7);
            const int row = min((h & 1) * 128 + r, (h < 2 ? a.N - n0 : a.M - m0) - 1);
            off[h][q] = static_cast<uint32_t>(row) * static_cast<uint32_t>(h < 2 ? a.wr : a.xr) + 16 * ch;
        }
    auto ask = [&](int k, int stage, int h) {
        const int kk = k < nk ? k : 0;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t o = off[h][q];
            if (TAIL && kk == nk - 1) {
                const int r = 16 * w + 8 * q + rl, ch = pc ^ (h < 2 ? keyA(r) : r & 7);
                o -= 16 * max(ch - (tail / 16 - 1), 0);
            }
            __builtin_amdgcn_raw_ptr_buffer_load_lds(h < 2 ? baseA : baseB,
                                                     (lds_void *)&sm[h >> 1][stage][h & 1][(16 * w + 8 * q) * BK], 16, o,
                                                     kk * BK, 0, 0);
        }
    };
    const int ra = 64 * wr + 8 * (c >> 2) + (c & 3);  // A's row of tile 0
    const int rb = 32 * wc + c;                         // B's row of tile 0 (tile s: + 16 s)
    const int8_t *pa[2], *pb[2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
        pa[kk] = &sm[0][0][0][ra * BK + 16 * ((4 * kk + g) ^ (c & 7))];  // keyA of A's rows is c & 7
        pb[kk] = &sm[1][0][0][rb * BK + 16 * ((4 * kk + g) ^ (c & 7))];
    }
    auto read_a = [&](int stage, int h, i32x4 (&f)[2][4]) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                f[kk][t] = *reinterpret_cast<const i32x4 *>(pa[kk] + (2 * stage + h) * 128 * BK + (32 * (t / 2) + 4 * (t % 2)) * BK);
    };
    auto read_b = [&](int stage, int h, i32x4 (&f)[2][2]) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                f[kk][s] = *reinterpret_cast<const i32x4 *>(pb[kk] + (2 * stage + h) * 128 * BK + 16 * s * BK);
    };
    auto cut = [&](int k, i32x4 (&f)[2][4]) {  // past K
        if (TAIL && k == nk - 1) {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (16 * (4 * kk + g) >= tail) f[kk][t] = i32x4{0, 0, 0, 0};
        }
    };
    i32x4 acc[2][2][4][2] = {};  // quadrant (A half, B half), tiles
    auto multiply = [&](i32x4 (&q)[4][2], const i32x4 (&fa)[2][4], const i32x4 (&fb_)[2][2]) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int s = 0; s < 2; ++s) q[t][s] = mfma_i8(fa[kk][t], fb_[kk][s], q[t][s]);
        __builtin_amdgcn_s_setprio(0);
        section_end();
    };
    auto m_end = [&] {
        fence();
        __builtin_amdgcn_s_waitcnt(0x0F70 | 12);  // vmcnt(12)
        __builtin_amdgcn_s_waitcnt(0xC07F);       // lgkmcnt(0)
        section_end();
    };
    i32x4 a0[2][4], a1[2][4], b0[2][2], b1[2][2];
    // A0 A1 B0 B1 are halves 0 1 2 3, asked for in the order 2 0 1 3
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        ask(k, k, 2);
        ask(k, k, 0);
        ask(k, k, 1);
        ask(k, k, 3);
    }
    m_end();  // the first halves 2 and 0
    read_b(0, 0, b0);
    m_end();
    if (wr) section_end();
    auto step = [&](int k, int stage) {
        read_a(stage, 0, a0);
        ask(k + 2, stage, 2);
        cut(k, a0);
        m_end();
        multiply(acc[0][0], a0, b0);
        read_a(stage, 1, a1);
        ask(k + 2, stage, 0);
        cut(k, a1);
        m_end();
        multiply(acc[1][0], a1, b0);
        read_b(stage, 1, b1);
        ask(k + 2, stage, 1);
        m_end();
        multiply(acc[1][1], a1, b1);
        read_b(stage ^ 1, 0, b0);
        ask(k + 2, stage, 3);
        m_end();
        multiply(acc[0][1], a0, b1);
    };
    for (int k = 0; k < nk; k += 2) {
        step(k, 0);
        if (k + 1 < nk) step(k + 1, 1);
    }
    if (!wr) section_end();
    // all scales at once, with the loads behind the last step
    const Lanes f[2] = {{a, n0 + 64 * wr + 8 * g}, {a, n0 + 128 + 64 * wr + 8 * g}};
    float sx[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s) sx[j][s] = a.xs[min(m0 + 128 * j + 32 * wc + 16 * s + c, a.M - 1)];
    __builtin_amdgcn_s_waitcnt(0x0F70);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                store16(a, m0 + 128 * j + 32 * wc + 16 * s + c, n0 + 128 * i + 64 * wr + 8 * g, sx[j][s], f[i],
                        [&](int t) { return acc[i][j][t][s]; });
}

// bytes of a row of K in LDS: whole steps, and 16 more so that rows start in other banks
inline int few_stride(int K) { return (K + 63) / 64 * 64 + 16; }

bool aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// whole 16-byte chunks, at 16-byte addresses
bool chunked(const int8_t *p, int64_t stride, int K) { return K % 16 == 0 && stride % 16 == 0 && aligned(p); }

void outputs(I8Args &a) { a.vec = a.H || (aligned(a.y) && a.yr * (a.out_io ? 2 : 4) % 16 == 0); }

template <int FT, int MT> hipError_t few(const I8Args &a, hipStream_t s) {
    const dim3 grid((a.N + 16 * FT - 1) / (16 * FT));
    if (chunked(a.x, a.xr, a.K) && chunked(a.w, a.wr, a.K))
        hipLaunchKernelGGL((i8_few<FT, MT, true>), grid, dim3(64 * FW), 0, s, a);
    else
        hipLaunchKernelGGL((i8_few<FT, MT, false>), grid, dim3(64 * FW), 0, s, a);
    return hipGetLastError();
}

template <typename T> hipError_t few_features(const I8Args &a, const void *in, int64_t xr, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const T *x = static_cast<const T *>(in);
    const bool vec = a.K % V == 0 && xr % V == 0 && aligned(x), chunks = chunked(a.w, a.wr, a.K);
    int W = 64 * FW;  // threads a row
    while (W > 64 && (64 * FW / W) < a.M) W /= 2;
    const int stride = few_stride(a.K);
    const dim3 grid((a.N + 15) / 16);
    const size_t lds = static_cast<size_t>(a.M) * stride;
    if (vec && chunks)
        hipLaunchKernelGGL((i8_few_features<T, V, true>), grid, dim3(64 * FW), lds, s, a, x, xr, W, stride);
    else
        hipLaunchKernelGGL((i8_few_features<T, 1, false>), grid, dim3(64 * FW), lds, s, a, x, xr, W, stride);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_i8_project(const I8Args &in, hipStream_t s) {
    I8Args a = in;
    outputs(a);
    if (a.M <= 16) return few<1, 1>(a, s);
    if (a.M <= 32) return few<1, 2>(a, s);
    if (a.M <= 64) return a.N >= 4096 ? few<2, 4>(a, s) : few<1, 4>(a, s);
    const bool big = chunked(a.x, a.xr, a.K) && chunked(a.w, a.wr, a.K) && a.xr < (1 << 23) && a.wr < (1 << 23);  // offsets in 32 bits
    const int nfb = (a.N + BT - 1) / BT, ntb = (a.M + BT - 1) / BT;
    if (big) {
        const dim3 grid(static_cast<unsigned>(nfb * ntb));
        if (a.K % BK)
            hipLaunchKernelGGL(i8_big<true>, grid, dim3(512), 0, s, a, nfb, ntb);
        else
            hipLaunchKernelGGL(i8_big<false>, grid, dim3(512), 0, s, a, nfb, ntb);
        return hipGetLastError();
    }
    const int64_t tiles = (static_cast<int64_t>(a.N) + GT - 1) / GT * ((static_cast<int64_t>(a.M) + GT - 1) / GT);
    hipLaunchKernelGGL(i8_any, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, s, a);
    return hipGetLastError();
}

// Up to 16 rows whose bytes fit beside the sums in 64 KB: one launch from the features.
bool i8_features_in_one(const I8Args &a) { return a.M <= 16 && static_cast<int64_t>(a.M) * few_stride(a.K) <= 48 * 1024; }

hipError_t launch_i8_features(const I8Args &in, int io, const void *x, int64_t xr, hipStream_t s) {
    I8Args a = in;
    outputs(a);
    return io ? few_features<bf16_t>(a, x, xr, s) : few_features<float>(a, x, xr, s);
}

}  // namespace ttt
