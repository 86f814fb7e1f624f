// The state space scan's backward, last part. The gradient of the log-decay
// l_t = D_t A of a token is q_t = <g_t, a_t h_{t-1}>, and from the two
// recurrences
//     q_t = q_{t+1} + dy_t . C_t (a_t h_{t-1}) - u_t . B_t (a_{t+1} g_{t+1}),
// so it is a running sum, from each segment's end backwards, of two per-token
// products that the walks have (row and col: both without the token's own
// term, which is in both and would only cancel), starting from the product of
// the state and its gradient at the segment's end. Sums run in 64 bits within
// a segment of at most 256 tokens. Then
//     ddt_t = (A q_t + x_t . du_t) sigma(dt_t + dt_bias),
//     dA = sum D_t q_t,  dD = sum dy_t . x_t,  ddt_bias = sum ddt_t,
// and dB, dC are summed over the heads of a group.
#include "block.hpp"
#include "ssm.hpp"
#include "vec.hpp"

namespace ttt {
namespace {

constexpr int NT = 256;

struct FinishArgs {
    SsmBwdArgs g;
    SsmBwdWs w;
    int brow, bcol;
};

__device__ __forceinline__ double block_sum(double v, double (&red)[NT / 64]) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    __syncthreads();
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

template <typename TIO>
__global__ __launch_bounds__(NT) void decay_gradient(FinishArgs f) {
    const SsmArgs &a = f.g.f;
    __shared__ double red[NT / 64], scan[2][NT];
    const int seg = blockIdx.x % a.nseg, bh = blockIdx.x / a.nseg, b = bh / a.H, h = bh % a.H;
    const int64_t NP = static_cast<int64_t>(a.N) * a.P;
    const int n = a.lens ? max(0, min(a.lens[b], a.L)) : a.L;
    const int64_t t = static_cast<int64_t>(seg) * a.seglen + threadIdx.x;
    const bool mine = static_cast<int>(threadIdx.x) < a.seglen && t < a.L, live = mine && t < n;
    // <state, its gradient> at the segment's end
    const float *se = seg + 1 < a.nseg ? f.w.sf + (static_cast<int64_t>(bh) * a.nseg + seg + 1) * NP : f.w.last + bh * NP;
    const float *ge = f.w.sr + (static_cast<int64_t>(bh) * a.nseg + seg) * NP;
    double e = 0.0;
    for (int64_t i = threadIdx.x; i < NP; i += NT) e += static_cast<double>(se[i]) * ge[i];
    e = block_sum(e, red);
    // sum over the tokens from this one to the segment's end
    const int64_t tok = static_cast<int64_t>(bh) * a.L + t, blk = static_cast<int64_t>(a.B) * a.H * a.L;
    double v = 0.0, xdu = 0.0, dyx = 0.0;
    if (live) {
        for (int i = 0; i < f.brow; ++i) v += f.w.row[i * blk + tok];
        for (int i = 0; i < f.bcol; ++i) {
            v -= f.w.col[i * blk + tok];
            xdu += f.w.xdu[i * blk + tok];
            dyx += f.w.dyx[i * blk + tok];
        }
    }
    int from = 0;
    scan[0][threadIdx.x] = v;
    __syncthreads();
#pragma unroll
    for (int m = 1; m < NT; m *= 2) {
        double s = scan[from][threadIdx.x];
        if (threadIdx.x + m < NT) s += scan[from][threadIdx.x + m];
        scan[from ^ 1][threadIdx.x] = s;
        from ^= 1;
        __syncthreads();
    }
    const double q = scan[from][threadIdx.x] + e;
    double dz = 0.0, dA = 0.0;
    if (live) {
        const float z = io_traits<TIO>::load(static_cast<const TIO *>(a.dt.p), b * a.dt.sb + t * a.dt.st + h * a.dt.sh) +
                        (a.dt_bias ? a.dt_bias[h] : 0.f);
        dA = q * softplus_f(z);
        dz = (a.A[h] * q + xdu) / (1.0 + exp(-static_cast<double>(z)));
    }
    if (mine)
        io_traits<TIO>::store(static_cast<TIO *>(const_cast<void *>(f.g.ddt.p)),
                              b * f.g.ddt.sb + t * f.g.ddt.st + h * f.g.ddt.sh, static_cast<float>(dz));
    dA = block_sum(dA, red);
    const double dD = block_sum(dyx, red), db = block_sum(dz, red);
    if (threadIdx.x == 0) {
        float *p = f.w.part + (static_cast<int64_t>(b) * a.nseg + seg) * 3 * a.H + h;
        p[0] = static_cast<float>(dA);
        p[a.H] = static_cast<float>(dD);
        p[2 * a.H] = static_cast<float>(db);
    }
}

// dB and dC from the heads' parts, a group's heads in order
template <typename TIO>
__global__ __launch_bounds__(NT) void head_sums(FinishArgs f) {
    const SsmArgs &a = f.g.f;
    const int64_t LN = static_cast<int64_t>(a.L) * a.N, all = a.B * a.G * LN;
    const int R = a.H / a.G;
    const bool second = blockIdx.y;
    const SsmOperand &o = second ? f.g.dC : f.g.dB;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * NT + threadIdx.x; i < all;
         i += static_cast<int64_t>(gridDim.x) * NT) {  // (b, g, t, n)
        const int n = static_cast<int>(i % a.N), t = static_cast<int>(i / a.N % a.L);
        const int g = static_cast<int>(i / LN % a.G), b = static_cast<int>(i / LN / a.G);
        const float *p = (second ? f.w.dCh : f.w.dBh) +
                         (static_cast<int64_t>(b) * a.H + static_cast<int64_t>(g) * R) * LN +
                         static_cast<int64_t>(t) * a.N + n;
        float s = 0.f;
        for (int r = 0; r < R; ++r) s += p[r * LN];
        io_traits<TIO>::store(static_cast<TIO *>(const_cast<void *>(o.p)), b * o.sb + t * o.st + g * o.sh + n, s);
    }
}

template <typename TIO> hipError_t finish(const FinishArgs &f, hipStream_t s) {
    const SsmArgs &a = f.g.f;
    const int64_t heads = static_cast<int64_t>(a.B) * a.H;
    hipError_t e = hipSuccess;
    if (heads) {
        hipLaunchKernelGGL((decay_gradient<TIO>), dim3(static_cast<unsigned>(heads * a.nseg)), dim3(NT), 0, s, f);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int64_t n = static_cast<int64_t>(a.B) * a.G * a.L * a.N;
    if (n) {
        const int64_t blocks = (n + NT - 1) / NT;
        hipLaunchKernelGGL((head_sums<TIO>), dim3(static_cast<unsigned>(blocks < (1 << 20) ? blocks : 1 << 20), 2),
                           dim3(NT), 0, s, f);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    ColumnSums c{f.w.part, 3 * static_cast<int64_t>(a.H), a.B * a.nseg};
    c.add(0, a.H, 1, f.g.dA);
    c.add(a.H, a.H, 1, f.g.dD);
    c.add(2 * static_cast<int64_t>(a.H), a.H, 1, f.g.ddt_bias);
    return launch_column_sums(c, s);
}

}  // namespace

SsmBwdWs ssm_backward_ws(const SsmArgs &a) {
    const int64_t BH = static_cast<int64_t>(a.B) * a.H, NP = static_cast<int64_t>(a.N) * a.P;
    SsmBwdWs w;
    w.floats = 0;
    auto take = [&](int64_t n) {
        float *q = a.ws ? a.ws + w.floats : nullptr;
        w.floats += static_cast<size_t>((n + 3) / 4 * 4);
        return q;
    };
    w.sf = take(BH * a.nseg * NP);
    w.sr = take(BH * a.nseg * NP);
    w.last = take(BH * NP);
    w.decay = take(BH * a.nseg);
    w.dBh = take(BH * a.L * a.N);
    w.dCh = take(BH * a.L * a.N);
    w.row = take(2 * BH * a.L);
    w.col = take(2 * BH * a.L);
    w.xdu = take(2 * BH * a.L);
    w.dyx = take(2 * BH * a.L);
    w.part = take(static_cast<int64_t>(a.B) * a.nseg * 3 * a.H);
    return w;
}

size_t ssm_backward_floats(int B, int L, int H, int P, int N, int nseg) {
    SsmArgs a{};
    a.B = B; a.L = L; a.H = H; a.P = P; a.N = N; a.nseg = nseg;
    return ssm_backward_ws(a).floats;
}

size_t ssm_forward_floats(int B, int H, int P, int N, int nseg) {
    return nseg > 1 ? static_cast<size_t>(B) * H * nseg * (static_cast<size_t>(N) * P + 1) : 0;
}

void ssm_segments(int B, int L, int H, int P, int N, bool mfma, bool backward, int *nseg, int *seglen) {
    (void)P;
    (void)mfma;
    // as many workgroups as run at once (three a compute unit, two where N
    // takes more of its LDS and registers), segments of whole 64-token chunks;
    // the backward's running sums over a segment hold at most 256 tokens
    const int64_t slots = N > 64 ? 512 : 768;
    const int64_t heads = static_cast<int64_t>(B) * H;
    const int64_t chunks = (static_cast<int64_t>(L) + 63) / 64;
    int64_t want = heads > 0 ? slots / heads : 1;
    if (want > chunks) want = chunks;
    if (want < 1) want = 1;
    int64_t per = (chunks + want - 1) / want;
    if (backward && per > 4) per = 4;
    if (per < 1) per = 1;
    *seglen = static_cast<int>(per * 64);
    *nseg = static_cast<int>(chunks > 0 ? (chunks + per - 1) / per : 1);
}

hipError_t launch_ssm_bwd_finish(const SsmBwdArgs &g, int blocks_row, int blocks_col, hipStream_t stream) {
    const FinishArgs f{g, ssm_backward_ws(g.f), blocks_row, blocks_col};
    return g.f.io == 1 ? finish<bf16_t>(f, stream) : finish<float>(f, stream);
}

}  // namespace ttt
