// 8-bit integer product with a scale for each token and each feature,
//     y[m][n] = xs[m] ws[n] sum_k x[m][k] w[n][k] (+ bias[n]),
// the sum exact in 32 bits (K <= 65536: below 2^30), then two products and a
// sum in fp32 and one rounding to y's type. Computed transposed, w as the A
// operand of the 16x16x64 MFMA, so that a lane's four accumulators are four
// consecutive features of one token.
#include "i8_scale.hpp"
#include "vec.hpp"

#include <algorithm>
#include <type_traits>

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

// Rows of K bytes at any address as rows of whole 128-byte lines, zeros past K: for
// operands that the large products could not read 16 bytes at a time. A wave a row.
// 16384 and 2048 rows of 2047: 14 us and the product 74, where reading them as they
// stand for each tile took 305; 1551 and 1037 rows of 771: 4.6 and 13.5, and 17.
__global__ __launch_bounds__(256) void i8_pad(I8PadArgs a) {
    const int lane = threadIdx.x & 63;
    int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int second = row >= a.rows[0];
    if (second) row -= a.rows[0];
    if (row >= a.rows[second]) return;
    const int8_t *src = a.src[second] + row * a.stride[second];
    int8_t *dst = a.dst[second] + row * a.pad;
    for (int k = lane * 16; k < a.pad; k += 1024) *reinterpret_cast<i32x4 *>(dst + k) = load16(src, k, a.K);
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

// Where logical chunk j of row r of a half lies among its eight: j ^ key(r). A's
// rows are a wave's TA MFMA tiles by pairs, 8 consecutive features of each pair to a
// lane; the last of an odd number of tiles goes by fours.
template <int TA> __device__ __forceinline__ int keyA(int r) {
    const int q = r % (16 * TA);
    return TA % 2 && q >= 16 * (TA - 1) ? q & 7 : (q & 3) | ((q >> 1) & 4);
}
// the row of MFMA row c of tile t, from a wave's first
template <int TA> constexpr __device__ __forceinline__ int rowA(int t, int c) {
    return TA % 2 && t == TA - 1 ? 16 * t + c : 32 * (t / 2) + 8 * (c >> 2) + 4 * (t % 2) + (c & 3);
}

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

// G = 8 or 4 consecutive features n .. of token m, whose scale is sx, where a.vec
template <int G>
__device__ __forceinline__ void store_run(const I8Args &a, int m, int n, float sx, const Features<G> &f, const i32x4 (&acc)[G / 4]) {
    if (m >= a.M || n >= a.N) return;
    float o[G];
#pragma unroll
    for (int e = 0; e < G; ++e) o[e] = fmaf(static_cast<float>(acc[e / 4][e % 4]) * sx, f.ws[e], f.bias[e]);
    const bool vec = n + G <= a.N;
    if (a.out_io) {
        // N is a multiple of 64 there: all of one head
        uint16_t *y = a.H ? view_at(a, m, n) : static_cast<uint16_t *>(a.y) + (m * a.yr + n);
        if (vec) {
            VecIO<bf16_t, G>::store(y, o);
        } else {
#pragma unroll
            for (int e = 0; e < G; ++e)
                if (n + e < a.N) y[e] = f32_to_bf16(o[e]);
        }
    } else {
        float *y = static_cast<float *>(a.y) + (m * a.yr + n);
        if (vec) {
            VecIO<float, G>::store(y, o);
        } else {
#pragma unroll
            for (int e = 0; e < G; ++e)
                if (n + e < a.N) y[e] = o[e];
        }
    }
}

// Large products: a workgroup of 8 waves takes 2 HA features x 2 HB tokens, 256 x
// 256 where there are tiles enough. Contraction steps of 128 bytes; both operands
// lie in LDS in halves of HA and HB rows, two stages, filled by direct
// global-to-LDS loads.
//  * a wave (wr, wc) takes HA / 2 x HB / 4 of each of the four quadrants (a half of
//    the features by a half of the tokens): TA x TB MFMA tiles, and walks them as
//    (0,0), (1,0), (1,1), (0,1), so that a step reads every fragment once;
//  * a quadrant is two sections: M reads the fragments that it or the next
//    quadrant lacks (2 TA or 2 TB of 1 KB) and asks for the half of two steps ahead
//    whose place was read last, C is its 2 TA TB products. A barrier ends each
//    section, and the waves 4 .. 7 run one section behind the waves 0 .. 3: on
//    each SIMD one wave multiplies while the other one reads;
//  * a half is asked for 7 M sections before it is read (in QA or QB loads of a
//    wave): s_waitcnt vmcnt at the end of M leaves the younger ones, 12 of them for
//    256 x 256, in flight. That wait and the one for the section's own LDS reads
//    stand before the section's barrier, so behind it every wave's loads have
//    landed, and the place of what was read may be filled again;
//  * rows of 128 bytes, 16-byte chunk j of row r at j ^ key(r): 8 distinct
//    places for the 8 rows that a fragment read touches at once. A's rows go to
//    MFMA rows so that a lane ends up with 8 consecutive features of a token (16
//    bytes of bf16) and a store of four lanes with 64 bytes;
//  * past K (TAIL) the last chunk is read again and A's is taken as zeros; rows past
//    the end are read from the last one and not stored.
// 16384 x 2048 x 6144: 178 us, 2.3 POP/s (a large library product in 8 bits: 2.1); a
// step takes 1.4 us, 0.97 with operands of zeros where 0.86 is the matrix cores' own
// at 2.4 GHz: what bounds it is the clock that the card holds under this load. A tile
// costs 7 to 9 us besides its steps (first loads, stores); walking over tiles with
// one workgroup a compute unit, the next tile's loads ahead, took as long.
constexpr int BK = 128;

typedef __attribute__((address_space(3))) void lds_void;

// Rows from p on, for loads by a 32-bit offset; the offsets stay within the rows.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const int8_t *p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(p), 0, 0xffffffff, 0x00027000);
}
__device__ __forceinline__ void fence() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void wave_order() {  // a wave's LDS accesses in the order that is written
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}
__device__ __forceinline__ void section_end() {  // barrier alone: no wait
    fence();
    __builtin_amdgcn_s_barrier();
    fence();
}

template <int HA, int HB, bool TAIL> __global__ __launch_bounds__(512, 2) void i8_big(I8Args a, int nfb, int ntb) {
    constexpr int TA = HA / 32, TB = HB / 64;
    constexpr int QA = (HA + 63) / 64, QB = (HB + 63) / 64;  // loads of a wave for a half, 8 rows each
    // [stage][half] of A, then of B: up to 64 KB each that one address reaches. One array: told two
    // apart, the compiler sees which loads to LDS a read may meet and waits for them all.
    constexpr int LA = HA * BK, LB = HB * BK;
    __shared__ __attribute__((aligned(16))) int8_t sm[4 * LA + 4 * LB];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4, c = lane & 15;
    const int wr = w >> 2, wc = w & 3;
    int fb, tb;
    tile_of(blockIdx.x, nfb, ntb, &fb, &tb);
    const int n0 = fb * 2 * HA, m0 = tb * 2 * HB;
    const int nk = (a.K + BK - 1) / BK, tail = TAIL ? a.K % BK : 0;  // a multiple of 16

    // loads: a wave's instruction q fills rows 8 (Q w + q) .. + 7 of a half (with HA = 96 the last
    // four of the sixteen rows that are asked for beyond it are others again)
    const auto baseA = buffer(a.w + static_cast<int64_t>(n0) * a.wr), baseB = buffer(a.x + static_cast<int64_t>(m0) * a.xr);
    const int rl = lane >> 3, pc = lane & 7;
    auto first = [&](bool isA, int q) { return isA ? 8 * (QA * w + q) % HA : 8 * (QB * w + q) % HB; };
    auto chunk = [&](bool isA, int q) {
        const int r = first(isA, q) + rl;
        return pc ^ (isA ? keyA<TA>(r) : r & 7);
    };
    uint32_t offA[2][QA], offB[2][QB];  // of the halves' rows from their base
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int q = 0; q < QA; ++q)
            offA[h][q] = static_cast<uint32_t>(min(h * HA + first(true, q) + rl, a.N - n0 - 1)) * static_cast<uint32_t>(a.wr) +
                         16 * chunk(true, q);
#pragma unroll
        for (int q = 0; q < QB; ++q)
            offB[h][q] = static_cast<uint32_t>(min(h * HB + first(false, q) + rl, a.M - m0 - 1)) * static_cast<uint32_t>(a.xr) +
                         16 * chunk(false, q);
    }
    auto ask = [&](int k, int stage, bool isA, int h) {
        const int kk = k < nk ? k : 0;  // behind the last step: the first again
#pragma unroll
        for (int q = 0; q < (isA ? QA : QB); ++q) {
            uint32_t o = isA ? offA[h][q < QA ? q : 0] : offB[h][q < QB ? q : 0];
            if (TAIL && kk == nk - 1) o -= 16 * max(chunk(isA, q) - (tail / 16 - 1), 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                isA ? baseA : baseB,
                (lds_void *)&sm[isA ? (2 * stage + h) * LA + first(true, q) * BK : 4 * LA + (2 * stage + h) * LB + first(false, q) * BK],
                16, o, kk * BK, 0, 0);
        }
    };
    const int8_t *pa[2], *pl[2], *pb[2];  // A's tiles by pairs, its last of an odd number, B's
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {  // the keys of MFMA rows c are c & 7
        const int j = 16 * ((4 * kk + g) ^ (c & 7));
        pa[kk] = &sm[(16 * TA * wr + rowA<TA>(0, c)) * BK + j];
        pl[kk] = &sm[(16 * TA * wr + c) * BK + j];
        pb[kk] = &sm[4 * LA + (16 * TB * wc + c) * BK + j];
    }
    auto read_a = [&](int stage, int h, i32x4 (&f)[2][TA]) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int t = 0; t < TA; ++t) {
                const bool last = TA % 2 && t == TA - 1;
                f[kk][t] = *reinterpret_cast<const i32x4 *>((last ? pl[kk] : pa[kk]) + (2 * stage + h) * LA +
                                                            (last ? 16 * t : rowA<TA>(t, 0)) * BK);
            }
    };
    auto read_b = [&](int stage, int h, i32x4 (&f)[2][TB]) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int s = 0; s < TB; ++s)
                f[kk][s] = *reinterpret_cast<const i32x4 *>(pb[kk] + (2 * stage + h) * LB + 16 * s * BK);
    };
    auto cut = [&](int k, i32x4 (&f)[2][TA]) {  // past K
        if (TAIL && k == nk - 1) {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int t = 0; t < TA; ++t)
                    if (16 * (4 * kk + g) >= tail) f[kk][t] = i32x4{0, 0, 0, 0};
        }
    };
    i32x4 acc[2][2][TA][TB] = {};  // quadrant (A half, B half), tiles
    auto multiply = [&](i32x4 (&q)[TA][TB], const i32x4 (&fa)[2][TA], const i32x4 (&fb_)[2][TB]) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int t = 0; t < TA; ++t)
#pragma unroll
                for (int s = 0; s < TB; ++s) q[t][s] = mfma_i8(fa[kk][t], fb_[kk][s], q[t][s]);
        __builtin_amdgcn_s_setprio(0);
        section_end();
    };
    // `young`: the loads asked for after the half that the next section reads
    auto m_end = [&](auto young) {
        fence();
        __builtin_amdgcn_s_waitcnt(0x0F70 | decltype(young)::value);  // vmcnt
        __builtin_amdgcn_s_waitcnt(0xC07F);                           // lgkmcnt(0)
        section_end();
    };
    static_assert(4 * QA + 2 * QB <= 15 && 2 * QA + 4 * QB <= 15, "counts of the low field");
    typedef std::integral_constant<int, 2 * QA + 4 * QB> Young0;
    typedef std::integral_constant<int, 3 * QA + 3 * QB> Young1;
    typedef std::integral_constant<int, 4 * QA + 2 * QB> Young2;
    i32x4 a0[2][TA], a1[2][TA], b0[2][TB], b1[2][TB];
    // the order of asking: B0 A0 A1 B1
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        ask(k, k, false, 0);
        ask(k, k, true, 0);
        ask(k, k, true, 1);
        ask(k, k, false, 1);
    }
    m_end(Young1{});  // the first B0 and A0
    read_b(0, 0, b0);
    m_end(Young1{});
    if (wr) section_end();
    auto step = [&](int k, int stage) {
        read_a(stage, 0, a0);
        ask(k + 2, stage, false, 0);
        cut(k, a0);
        m_end(Young0{});  // A1
        multiply(acc[0][0], a0, b0);
        read_a(stage, 1, a1);
        ask(k + 2, stage, true, 0);
        cut(k, a1);
        m_end(Young1{});  // B1
        multiply(acc[1][0], a1, b0);
        read_b(stage, 1, b1);
        ask(k + 2, stage, true, 1);
        m_end(Young2{});  // the next step's B0
        multiply(acc[1][1], a1, b1);
        read_b(stage ^ 1, 0, b0);
        ask(k + 2, stage, false, 1);
        m_end(Young1{});  // and A0
        multiply(acc[0][1], a0, b1);
    };
    for (int k = 0; k < nk; k += 2) {
        step(k, 0);
        if (k + 1 < nk) step(k + 1, 1);
    }
    if (!wr) section_end();
    // all scales at once, with the loads behind the last step
    float sx[2][TB];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int s = 0; s < TB; ++s) sx[j][s] = a.xs[min(m0 + HB * j + 16 * TB * wc + 16 * s + c, a.M - 1)];
    const int nw = n0 + 16 * TA * wr;
    // by pairs of tiles (the second pair, where there is one), and an odd tile's
    const Features<8> p0[2] = {Features<8>(a, nw + 8 * g), Features<8>(a, nw + HA + 8 * g)};
    const Features<8> p1[2] = {Features<8>(a, nw + 32 + 8 * g), Features<8>(a, nw + HA + 32 + 8 * g)};
    const Features<4> odd[2] = {Features<4>(a, nw + 16 * (TA - 1) + 4 * g), Features<4>(a, nw + HA + 16 * (TA - 1) + 4 * g)};
    __builtin_amdgcn_s_waitcnt(0x0F70);
    if (!a.vec) {  // outputs one by one: by way of LDS, so that a wave's lie side by side
        constexpr int F = 16 * TA, S = F + 4;
        __syncthreads();  // all waves' loads have landed
        float *const t = reinterpret_cast<float *>(sm) + w * 16 * S;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int s = 0; s < TB; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float *row = t + c * S;
#pragma unroll
                    for (int q = 0; q < TA; ++q) {
                        const bool last = TA % 2 && q == TA - 1;
                        const Features<8> &f = q / 2 ? p1[i] : p0[i];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            row[last ? 16 * q + 4 * g + e : 32 * (q / 2) + 8 * g + 4 * (q % 2) + e] =
                                fmaf(static_cast<float>(acc[i][j][q][s][e]) * sx[j][s], last ? odd[i].ws[e] : f.ws[4 * (q % 2) + e],
                                     last ? odd[i].bias[e] : f.bias[4 * (q % 2) + e]);
                    }
                    wave_order();
#pragma unroll
                    for (int e = 0; e < 16 * F / 64; ++e) {
                        const int at = 64 * e + lane, m = m0 + HB * j + 16 * TB * wc + 16 * s + at / F, n = nw + HA * i + at % F;
                        const float o = t[at / F * S + at % F];
                        if (m < a.M && n < a.N) {
                            if (a.out_io)
                                static_cast<uint16_t *>(a.y)[m * a.yr + n] = f32_to_bf16(o);
                            else
                                static_cast<float *>(a.y)[m * a.yr + n] = o;
                        }
                    }
                    wave_order();
                }
        return;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int s = 0; s < TB; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int m = m0 + HB * j + 16 * TB * wc + 16 * s + c, n = nw + HA * i;
#pragma unroll
                for (int p = 0; p < TA / 2; ++p)
                    store_run<8>(a, m, n + 32 * p + 8 * g, sx[j][s], p ? p1[i] : p0[i], {acc[i][j][2 * p][s], acc[i][j][2 * p + 1][s]});
                if constexpr (TA % 2 != 0)
                    store_run<4>(a, m, n + 16 * (TA - 1) + 4 * g, sx[j][s], odd[i], {acc[i][j][TA - 1][s]});
            }
}

template <int HA, int HB> hipError_t big(const I8Args &a, hipStream_t s) {
    const int nfb = (a.N + 2 * HA - 1) / (2 * HA), ntb = (a.M + 2 * HB - 1) / (2 * HB);
    const dim3 grid(static_cast<unsigned>(nfb * ntb));
    if (a.K % BK)
        hipLaunchKernelGGL((i8_big<HA, HB, true>), grid, dim3(512), 0, s, a, nfb, ntb);
    else
        hipLaunchKernelGGL((i8_big<HA, HB, false>), grid, dim3(512), 0, s, a, nfb, ntb);
    return hipGetLastError();
}

// bytes of a row of K in LDS: whole steps, and 16 more so that rows start in other banks
inline int few_stride(int K) { return (K + 63) / 64 * 64 + 16; }

bool aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// whole 16-byte chunks, at 16-byte addresses
bool chunked(const int8_t *p, int64_t stride, int K) { return K % 16 == 0 && stride % 16 == 0 && aligned(p); }

// and a tile's offsets in 32 bits
bool tileable(const int8_t *p, int64_t stride, int K) { return chunked(p, stride, K) && stride < (1 << 23); }

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

void i8_unaligned(const I8Args &a, bool *x, bool *w) {
    *x = a.M > 64 && !tileable(a.x, a.xr, a.K);
    *w = a.M > 64 && !tileable(a.w, a.wr, a.K);
}

hipError_t launch_i8_pad(const I8PadArgs &a, hipStream_t s) {
    const int64_t rows = static_cast<int64_t>(a.rows[0]) + a.rows[1];
    if (!rows) return hipSuccess;
    hipLaunchKernelGGL(i8_pad, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_i8_project(const I8Args &in, hipStream_t s) {
    I8Args a = in;
    outputs(a);
    if (a.M <= 16) return few<1, 1>(a, s);
    if (a.M <= 32) return few<1, 2>(a, s);
    // two tiles of features a workgroup where that still leaves half the compute units one: 64 x
    // 2048 x 6144 11.6 -> 8.6 us (a row of x is read half as often); below, one
    if (a.M <= 64) return a.N >= 4096 ? few<2, 4>(a, s) : few<1, 4>(a, s);
    // The tile shape whose rounds over the compute units take the least, by a step's time and a
    // tile's own (us, fitted to the measurements) in a full round and, for the last, alone on the
    // chip and in between. The smallest runs twice on a compute unit. Largest to smallest shape, 8192
    // tokens x 2304 features: K = 768 31.5, 30.2, 30.9, 28.7 us, K = 4096 89.6, 81.1, 89.3, 86.7;
    // 4096 x 4096 x 4096 58.0, 85.7, 74.8, 78.8; 4096 x 2048 x 4096 44.2, 42.2, 34.8, 36.8; 500 x 768 x 768
    // 13.4, 12.6, 9.2, 7.4. The model does not know outputs one by one (1551 x 784 x 1037 in bf16 12.7 us, x
    // 1040 9.5; in fp32 11.8 and 11.3), and K is not split: 128 x 8192 x 2048, 16 tiles of the smallest shape, 38.
    int dev = 0, ncu = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&ncu, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    const int steps = (a.K + BK - 1) / BK;
    struct Time { float step, tile; };
    auto us = [&](int f, int t, int at_once, Time full, Time alone) {
        const int64_t tiles = static_cast<int64_t>((a.N + f - 1) / f) * ((a.M + t - 1) / t);
        const float round = full.step * steps + full.tile, least = alone.step * steps + alone.tile;
        const int64_t rest = tiles % at_once;
        return static_cast<float>(tiles / at_once) * round + (rest ? least + (round - least) * rest / at_once : 0.f);
    };
    const float t0 = us(256, 256, ncu, {1.45f, 7.f}, {.89f, 6.f}), t1 = us(192, 256, ncu, {1.f, 7.6f}, {.82f, 6.5f}),
                t2 = us(128, 256, ncu, {.75f, 4.5f}, {.63f, 4.2f}), t3 = us(128, 128, 2 * ncu, {.74f, 4.9f}, {.51f, 3.5f});
    const float least = std::min(std::min(t0, t1), std::min(t2, t3));
    return least == t0 ? big<128, 128>(a, s) : least == t1 ? big<96, 128>(a, s) : least == t2 ? big<64, 128>(a, s) : big<64, 64>(a, s);
}

// Up to 16 rows whose bytes fit beside the sums in 64 KB: one launch from the features.
bool i8_features_in_one(const I8Args &a) { return a.M <= 16 && static_cast<int64_t>(a.M) * few_stride(a.K) <= 48 * 1024; }

hipError_t launch_i8_features(const I8Args &in, int io, const void *x, int64_t xr, hipStream_t s) {
    I8Args a = in;
    outputs(a);
    return io ? few_features<bf16_t>(a, x, xr, s) : few_features<float>(a, x, xr, s);
}

}  // namespace ttt
