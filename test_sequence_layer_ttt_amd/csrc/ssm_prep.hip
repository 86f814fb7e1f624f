// The decays of every 64-token chunk for the MFMA kernels: with D_t =
// softplus(dt_t + dt_bias), log2 of the decay since the chunk's start (in two
// floats), D_t and the decay to the chunk's end, 256 floats a chunk and head.
// They are the same for every wave and every pass over the chunk; made here
// once, the walks' first wave need not make them while the others wait.
// Bound by latency: 16 bytes out for each token and head; 5.9 us for 2 x 8192
// tokens and 32 heads, of which 8.4 MB written are 1.8.
#include "ssm_tile.hpp"

namespace ttt {
namespace {

using namespace ssm;

template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_add64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xF, true);
    return v + __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
// Inclusive sums over the lanes 0 .. lane: within rows of 16 lanes, then the
// rows' totals.
__device__ __forceinline__ double wave_scan(double v) {
    v = dpp_add64<0x111, 0xF>(v);  // row_shr:1
    v = dpp_add64<0x112, 0xF>(v);  // row_shr:2
    v = dpp_add64<0x114, 0xF>(v);  // row_shr:4
    v = dpp_add64<0x118, 0xF>(v);  // row_shr:8
    v = dpp_add64<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
    v = dpp_add64<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
    return v;
}


// A workgroup takes a chunk of HB heads: dt goes through LDS, so that its rows
// (heads adjacent) are read whole; then a wave takes a head, lane = token.
constexpr int HB = 16;
__global__ __launch_bounds__(64 * HB) void decays(SsmArgs a, int nch, float *out) {
    __shared__ float dts[Q][HB + 1];
    const int hb = (a.H + HB - 1) / HB;
    const int h0 = static_cast<int>(blockIdx.x % hb) * HB, bc = static_cast<int>(blockIdx.x / hb);
    const int c = bc % nch, b = bc / nch;
    const int lane = threadIdx.x % 64, t0 = c * Q;
    const int n = a.lens ? max(0, min(a.lens[b], a.L)) : a.L;
    const bf16_t *dt = static_cast<const bf16_t *>(a.dt.p) + b * a.dt.sb;
    const int t = threadIdx.x / HB, e = threadIdx.x % HB;
    if (t0 + t < n && h0 + e < a.H) dts[t][e] = bf16_to_f32(dt[static_cast<int64_t>(t0 + t) * a.dt.st + (h0 + e) * a.dt.sh]);
    __syncthreads();
    const int i = threadIdx.x / 64, h = h0 + i;
    if (h < a.H) {
        // Tokens past the sequence's end decay nothing and add nothing. A factor
        // below 2^-160 is zero in fp32 as it is, so logarithms are held above that.
        float step = 0.f;
        double l = 0.0;
        if (t0 + lane < n) {
            step = softplus_f(dts[lane][i] + (a.dt_bias ? a.dt_bias[h] : 0.f));
            l = at_least(static_cast<double>(step) * a.A[h] * 1.4426950408889634, -160.0);
        }
        const double s = wave_scan(l);
        const double all = __shfl(s, 63, 64);
        const float hi = static_cast<float>(s);
        float *o = out + (static_cast<int64_t>(b * a.H + h) * nch + c) * 4 * Q + lane;
        o[0] = hi;
        o[Q] = static_cast<float>(s - hi);
        o[2 * Q] = step;
        o[3 * Q] = __builtin_amdgcn_exp2f(static_cast<float>(all - s));
    }
}

}  // namespace

size_t ssm_prep_floats(int B, int L, int H) {
    return static_cast<size_t>(B) * H * ((static_cast<size_t>(L) + Q - 1) / Q) * 4 * Q;
}

hipError_t launch_ssm_prep(const SsmArgs &a, float *out, hipStream_t stream) {
    const int nch = static_cast<int>((static_cast<int64_t>(a.L) + Q - 1) / Q);
    const int64_t blocks = static_cast<int64_t>(a.B) * nch * ((a.H + HB - 1) / HB);
    if (!blocks) return hipSuccess;
    hipLaunchKernelGGL(decays, dim3(static_cast<unsigned>(blocks)), dim3(64 * HB), 0, stream, a, nch, out);
    return hipGetLastError();
}

}  // namespace ttt
