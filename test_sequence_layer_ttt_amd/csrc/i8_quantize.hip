// Rows of fp32 or bf16 in 8 bits: scale = max |x| / 127 in fp32 and
// q = x / scale rounded to the nearest whole number, ties to even, of the
// exact quotient, held to -127 .. 127.
//
// The quotient is not divided out: q0 = rint(x rcp(scale)) is the nearest
// whole number or one beside it, r = x - q0 scale is exact in one fused step
// (where |x| >= scale both are multiples of scale's last place; where it is
// not, q0 is 0 or r is a difference of numbers within a factor of two), and
// r against scale / 2 says which. Scales below 2^-120, where the reciprocal or
// the half could leave fp32's range, are divided in 64 bits.
//
// A row that holds an infinity or a NaN has a NaN for its scale and zeros for
// q, so that its products are NaN.
#include "i8.hpp"
#include "vec.hpp"

namespace ttt {
namespace {

constexpr int NT = 256;

__device__ __forceinline__ int nearest(float x, float s, float inv, float half) {
    float q = __builtin_rintf(x * inv);
    const float r = fmaf(-q, s, x);
    const bool odd = static_cast<int>(q) & 1;
    if (r > half || (r == half && odd)) q += 1.0f;
    if (r < -half || (r == -half && odd)) q -= 1.0f;
    return static_cast<int>(fminf(fmaxf(q, -127.0f), 127.0f));
}
__device__ __forceinline__ int nearest_small(float x, float s) {
    const double q = s > 0.f ? __builtin_rint(static_cast<double>(x) / static_cast<double>(s)) : 0.0;
    return static_cast<int>(fmin(fmax(q, -127.0), 127.0));
}

// One row to W threads. V values of 16 bytes at a time; a row is read twice,
// the second time from the chip's caches.
template <typename T, int V, int W>
__global__ __launch_bounds__(NT) void quantize(I8QuantArgs a) {
    __shared__ uint32_t red[NT / 64];
    const int lane = threadIdx.x % W;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * (NT / W) + threadIdx.x / W;
    const bool in = m < a.M;
    const T *x = static_cast<const T *>(a.x) + (in ? m : 0) * a.xr;
    uint32_t most = 0;  // bits of |x|: a NaN's are above an infinity's, these above all others
    if (in) {
        for (int k = lane * V; k < a.K; k += W * V) {
            float v[V];
            vec_load<T, V>(x + k, v);
#pragma unroll
            for (int e = 0; e < V; ++e) most = max(most, __float_as_uint(v[e]) & 0x7fffffffu);
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), d)));
    if constexpr (W > 64) {
        red[threadIdx.x / 64] = most;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) most = max(most, red[i]);
    }
    if (!in) return;
    const bool finite = most < 0x7f800000u;
    const float s = finite ? __uint_as_float(most) / 127.0f : __uint_as_float(0x7fc00000u);
    if (lane == 0) a.scale[m] = s;
    int8_t *q = a.q + m * a.qr;
    const float inv = __builtin_amdgcn_rcpf(s), half = 0.5f * s;
    for (int k = lane * V; k < a.K; k += W * V) {
        float v[V];
        vec_load<T, V>(x + k, v);
        int p[V];
#pragma unroll
        for (int e = 0; e < V; ++e)
            p[e] = !finite ? 0 : s >= 0x1p-120f ? nearest(v[e], s, inv, half) : nearest_small(v[e], s);
        if constexpr (V >= 4) {
#pragma unroll
            for (int e = 0; e < V; e += 4)
                *reinterpret_cast<uint32_t *>(q + k + e) = (p[e] & 255) | (p[e + 1] & 255) << 8 | (p[e + 2] & 255) << 16 |
                                                           static_cast<uint32_t>(p[e + 3]) << 24;
        } else {
            q[k] = static_cast<int8_t>(p[0]);
        }
    }
}

template <typename T, int V> hipError_t rows(const I8QuantArgs &a, hipStream_t s) {
    // a wave a row where that fills the chip or a row is no more than a wave's one load
    const bool wave = a.M >= 4096 || a.K <= 64 * V;
    const int64_t per = wave ? NT / 64 : 1;
    const dim3 grid(static_cast<unsigned>((a.M + per - 1) / per));
    if (wave)
        hipLaunchKernelGGL((quantize<T, V, 64>), grid, dim3(NT), 0, s, a);
    else
        hipLaunchKernelGGL((quantize<T, V, NT>), grid, dim3(NT), 0, s, a);
    return hipGetLastError();
}

template <typename T> hipError_t typed(const I8QuantArgs &a, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = a.K % V == 0 && a.xr % V == 0 && a.qr % 4 == 0 && (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 &&
                     (reinterpret_cast<uintptr_t>(a.q) & 3) == 0;
    return vec ? rows<T, V>(a, s) : rows<T, 1>(a, s);
}

}  // namespace

hipError_t launch_i8_quantize(const I8QuantArgs &a, hipStream_t s) {
    return a.io ? typed<bf16_t>(a, s) : typed<float>(a, s);
}

}  // namespace ttt
