// 8-bit integer product with a scale for each token and each feature,
//     y[m][n] = xs[m] ws[n] sum_k x[m][k] w[n][k] (+ bias[n]),
// the sum exact in 32 bits (K <= 65536: below 2^30), then two products and a
// sum in fp32 and one rounding to y's type. Computed transposed, w as the A
// operand of the 16x16x64 MFMA, so that a lane's four accumulators are four
// consecutive features of one token.
#include "i8.hpp"
#include "tile.hpp"

namespace ttt {
namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4;

__device__ __forceinline__ i32x4 mfma_i8(i32x4 a, i32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// Bytes k .. k + 15 of a row of K at any address, zeros from K on: the aligned
// words that hold one of them, shifted together. Every word that is read holds
// a byte of the row.
__device__ __forceinline__ i32x4 load16(const int8_t *row, int k, int K) {
    uint32_t d[5] = {};
    if (k < K) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(row + k), end = reinterpret_cast<uintptr_t>(row + K);
        const uint32_t *q = reinterpret_cast<const uint32_t *>(p & ~static_cast<uintptr_t>(3));
#pragma unroll
        for (int j = 0; j < 5; ++j)
            if (reinterpret_cast<uintptr_t>(q + j) < end) d[j] = q[j];
        const uint32_t sh = static_cast<uint32_t>(p & 3);
        const int live = K - k;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = __builtin_amdgcn_alignbyte(d[j + 1], d[j], sh);
            const int n = live - 4 * j;
            d[j] = n >= 4 ? v : n <= 0 ? 0u : v & ((1u << (8 * n)) - 1);
        }
    }
    return i32x4{static_cast<int>(d[0]), static_cast<int>(d[1]), static_cast<int>(d[2]), static_cast<int>(d[3])};
}

// features n .. n + 3 of token m
__device__ __forceinline__ void store4(const I8Args &a, int m, int n, i32x4 acc) {
    if (m >= a.M || n >= a.N) return;
    const float sx = a.xs[m];
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int f = min(n + e, a.N - 1);
        o[e] = static_cast<float>(acc[e]) * sx * a.ws[f];
        if (a.bias) o[e] += a.bias[f];
    }
    if (a.H) {  // N is a multiple of 64: four features of one head
        const int HD = a.H * 64, v = n / HD, hj = n - v * HD, b = m / a.L, t = m - b * a.L;
        uint16_t *out = static_cast<uint16_t *>(v == 0 ? a.v[0] : v == 1 ? a.v[1] : a.v[2]);
        out += ((static_cast<int64_t>(b) * a.H + hj / 64) * a.L + t) * 64 + hj % 64;
        *reinterpret_cast<uint2 *>(out) = make_uint2(tile::pack2(o[0], o[1]), tile::pack2(o[2], o[3]));
        return;
    }
    const int64_t at = m * a.yr + n;
    if (a.out_io) {
        uint16_t *y = static_cast<uint16_t *>(a.y) + at;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < a.N) y[e] = f32_to_bf16(o[e]);
    } else {
        float *y = static_cast<float *>(a.y) + at;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < a.N) y[e] = o[e];
    }
}

// Any sizes, strides and addresses: a workgroup takes 64 features x 64 tokens,
// a wave 32 x 32 of them, contraction steps of 64 bytes through LDS. Rows of
// 80 bytes: the 16 rows of a fragment read lie in distinct banks.
constexpr int GT = 64, GK = 64, GS = 80;

__global__ __launch_bounds__(256) void i8_any(I8Args a) {
    __shared__ __attribute__((aligned(16))) int8_t sw[GT * GS], sx[GT * GS];
    const int nf = (a.N + GT - 1) / GT;
    const int n0 = static_cast<int>(blockIdx.x % nf) * GT, m0 = static_cast<int>(blockIdx.x / nf) * GT;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, c = lane & 15;
    const int row = tid >> 2, part = (tid & 3) * 16;
    // rows behind the last are read from it; their outputs are not stored
    const int8_t *pw = a.w + static_cast<int64_t>(min(n0 + row, a.N - 1)) * a.wr;
    const int8_t *px = a.x + static_cast<int64_t>(min(m0 + row, a.M - 1)) * a.xr;
    const int wf = (w & 1) * 32, wt = (w >> 1) * 32;
    i32x4 acc[2][2] = {};
    i32x4 nw = load16(pw, part, a.K), nx = load16(px, part, a.K);
    for (int k = 0; k < a.K; k += GK) {
        *reinterpret_cast<i32x4 *>(&sw[row * GS + part]) = nw;
        *reinterpret_cast<i32x4 *>(&sx[row * GS + part]) = nx;
        __syncthreads();
        nw = load16(pw, k + GK + part, a.K);
        nx = load16(px, k + GK + part, a.K);
        i32x4 fw[2], fx[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            fw[i] = *reinterpret_cast<const i32x4 *>(&sw[(wf + 16 * i + c) * GS + 16 * g]);
            fx[i] = *reinterpret_cast<const i32x4 *>(&sx[(wt + 16 * i + c) * GS + 16 * g]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mfma_i8(fw[i], fx[j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) store4(a, m0 + wt + 16 * j + c, n0 + wf + 16 * i + 4 * g, acc[i][j]);
}

}  // namespace

hipError_t launch_i8_project(const I8Args &a, hipStream_t s) {
    const int64_t tiles = (static_cast<int64_t>(a.N) + GT - 1) / GT * ((static_cast<int64_t>(a.M) + GT - 1) / GT);
    hipLaunchKernelGGL(i8_any, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace ttt
