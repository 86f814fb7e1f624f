// Rows of fp32 or bf16 in 8 bits (the mathematics: i8_scale.hpp). HBM bound: a row
// is read once and held while its largest value is found.
#include "i8_scale.hpp"
#include "vec.hpp"

namespace ttt {
namespace {

constexpr int NT = 256;

// A grid's threads are counted in 32 bits along each of its dimensions: 2^24 rows of a
// workgroup each would be 2^32, so the workgroups go on in the second dimension after MOST.
constexpr int MOST = 1 << 22;

// One row to W threads, V values of 16 bytes (or one) at a time. R: the row is
// held in R of them a thread and read once; R = 0: of any length, read twice (the
// second time from the chip's caches).
template <typename T, int V, int W, int R>
__global__ __launch_bounds__(NT) void quantize(I8QuantArgs a) {
    typedef VecIO<T, V> IO;
    __shared__ uint32_t red[NT / 64];
    const int lane = threadIdx.x % W;
    const int64_t m = (static_cast<int64_t>(blockIdx.y) * MOST + blockIdx.x) * (NT / W) + threadIdx.x / W;
    if (m >= a.M) return;  // whole waves, and with W > 64 whole workgroups
    const T *x = static_cast<const T *>(a.x) + m * a.xr;
    int8_t *q = a.q + m * a.qr;
    uint32_t most = 0;  // bits of |x|: a NaN's are above an infinity's, these above all others
    auto look = [&](const typename IO::Raw &r) {
        float v[V];
        IO::unpack(r, v);
#pragma unroll
        for (int e = 0; e < V; ++e) most = max(most, __float_as_uint(v[e]) & 0x7fffffffu);
    };
    auto put = [&](const Scale &s, const typename IO::Raw &r, int k) {
        float v[V];
        IO::unpack(r, v);
        s.put<V>(v, q + k);
    };
    typename IO::Raw held[R ? R : 1];
    if constexpr (R > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int k = (i * W + lane) * V;
            held[i] = k < a.K ? IO::raw(x + k) : IO::zero();
        }
#pragma unroll
        for (int i = 0; i < R; ++i) look(held[i]);
    } else {
        for (int k = lane * V; k < a.K; k += W * V) look(IO::raw(x + k));
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), d)));
    if constexpr (W > 64) {
        red[threadIdx.x / 64] = most;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) most = max(most, red[i]);
    }
    const Scale s(most);
    if (lane == 0) a.scale[m] = s.s;
    if constexpr (R > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int k = (i * W + lane) * V;
            if (k < a.K) put(s, held[i], k);
        }
    } else {
        for (int k = lane * V; k < a.K; k += W * V) put(s, IO::raw(x + k), k);
    }
}

template <typename T, int V, int W, int R> hipError_t go(const I8QuantArgs &a, hipStream_t s) {
    const int64_t per = NT / W, n = (a.M + per - 1) / per;
    const dim3 grid(static_cast<unsigned>(n < MOST ? n : MOST), static_cast<unsigned>((n + MOST - 1) / MOST));
    hipLaunchKernelGGL((quantize<T, V, W, R>), grid, dim3(NT), 0, s, a);
    return hipGetLastError();
}

template <typename T, int V> hipError_t rows(const I8QuantArgs &a, hipStream_t s) {
    // A wave a row where that fills the chip (or the row is no more than a wave's one load), four
    // otherwise. 16384 rows of K = 2048 in bf16: 20.1 us (5.0 TB/s, a large copy's rate), 25.8 with the
    // borders looked at value by value, 28.7 with the row read twice.
    if (a.K <= 64 * V) return go<T, V, 64, 1>(a, s);
    if (a.M >= 2048 && a.K <= 64 * V * 2) return go<T, V, 64, 2>(a, s);
    if (a.M >= 2048 && a.K <= 64 * V * 4) return go<T, V, 64, 4>(a, s);
    if (a.K <= NT * V) return go<T, V, NT, 1>(a, s);
    if (a.K <= NT * V * 4) return go<T, V, NT, 4>(a, s);
    return go<T, V, NT, 0>(a, s);
}

template <typename T> hipError_t typed(const I8QuantArgs &a, hipStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = a.K % V == 0 && a.xr % V == 0 && a.qr % V == 0 && (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 &&
                     (reinterpret_cast<uintptr_t>(a.q) & (V - 1)) == 0;
    return vec ? rows<T, V>(a, s) : rows<T, 1>(a, s);
}

}  // namespace

hipError_t launch_i8_quantize(const I8QuantArgs &a, hipStream_t s) {
    return a.io ? typed<bf16_t>(a, s) : typed<float>(a, s);
}

}  // namespace ttt
