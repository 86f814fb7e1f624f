// The seam between two blocks of a layer stack: the norm after a block, its
// gate, the residual sum and the norm before the next block.
//     n  = Norm(y) post_gamma (+ post_beta)
//     r' = scale resid + act(gate) n
//     x  = Norm(r') pre_gamma (+ pre_beta)
// with Norm(u) = u / sqrt(mean u^2 + eps) or (u - mean u) / sqrt(var u + eps).
//
// HBM bound: a row's resid, y and gate are read once, r' and x written once.
// TPR threads hold a row in registers (64: one wave a row, no barriers; 256:
// a workgroup a row), the statistics are sums of registers (of centred values,
// so a common offset of the row costs no digits), and the next row's loads
// are issued before this row's sums are waited for. B=2 L=8192 D=2048, bf16 with
// an fp32 residual: 470 MB in 84 us, 5.6 TB/s; one token of D=768: 3.7 us, a
// launch and two dependent sums.
#include "block_norm.hpp"

namespace ttt {
namespace {

using namespace norm;

// One row's inputs, fetched ahead
template <class C, typename TIO, typename TR> struct RowIn {
    typename C::template Raws<TR> resid;
    typename C::template Raws<TIO> y, gate;
    bool live;
};

template <int TPR, int VEC, int NV, typename TIO, typename TR>
__global__ __launch_bounds__(threads(TPR)) void block_norm_fwd(NormArgs a, int rows) {
    typedef Cols<TPR, VEC, NV> C;
    constexpr int E = C::E, RPW = threads(TPR) / TPR;
    constexpr bool HOLD = E <= 16;  // parameters in registers over all rows
    __shared__ float red[4][threads(TPR) / 64];
    RowSum<TPR> sum{red};
    const C c{a.D, static_cast<int>(threadIdx.x % TPR)};
    const float inv_d = 1.0f / static_cast<float>(a.D);
    const int step = gridDim.x * RPW;
    float pg[E], pb[E], qg[E], qb[E], sc[E];
    if constexpr (HOLD) {
        c.param(a.post_gamma, 1.f, pg);
        c.param(a.post_beta, 0.f, pb);
        c.param(a.pre_gamma, 1.f, qg);
        c.param(a.pre_beta, 0.f, qb);
        c.param(a.scale, 1.f, sc);
    }
    auto fetch = [&](int row, RowIn<C, TIO, TR> &in) {
        const int b = row / a.L, t = row - b * a.L;
        in.live = !a.lens || t < a.lens[b];
        if (!in.live) return;
        c.fetch(static_cast<const TR *>(a.resid) + b * a.rb + t * a.rt, in.resid);
        c.fetch(static_cast<const TIO *>(a.y) + b * a.yb + t * a.yt, in.y);
        if (a.gmode == TTT_GATE_TOKEN) c.fetch(static_cast<const TIO *>(a.gate) + b * a.gb + t * a.gt, in.gate);
    };
    int row = blockIdx.x * RPW + threadIdx.x / TPR;
    RowIn<C, TIO, TR> in;
    if (row < rows) fetch(row, in);
    for (; row < rows; row += step) {
        TR *ro = static_cast<TR *>(a.resid_out) + static_cast<int64_t>(row) * a.D;
        TIO *xo = static_cast<TIO *>(a.x) + static_cast<int64_t>(row) * a.D;
        const bool live = in.live;
        float n[E], r[E], g[E];
        if (live) {
            c.unpack(in.y, n);
            c.unpack(in.resid, r);
            if (a.gmode == TTT_GATE_TOKEN) c.unpack(in.gate, g);
        }
        if (row < rows - step) fetch(row + step, in);
        if (!live) {  // past the sequence's end: zeros
#pragma unroll
            for (int e = 0; e < E; ++e) n[e] = 0.f;
            c.store(ro, n);
            c.store(xo, n);
            continue;
        }
        if (a.gmode == TTT_GATE_CHANNEL) c.load(static_cast<const float *>(a.gate), g);
        if (a.gmode == TTT_GATE_SEQUENCE)
            c.load(static_cast<const float *>(a.gate) + static_cast<int64_t>(row / a.L) * a.D, g);
        c.hat(n, a.layer, a.eps, inv_d, sum);
        if constexpr (!HOLD) {
            c.param(a.post_gamma, 1.f, pg);
            c.param(a.post_beta, 0.f, pb);
            c.param(a.scale, 1.f, sc);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) n[e] = fmaf(n[e], pg[e], pb[e]);
        if (a.gmode != TTT_GATE_NONE) {
            float v[E], dv[E];
            activate(a.act, g, v, dv);
#pragma unroll
            for (int e = 0; e < E; ++e) n[e] *= v[e];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = fmaf(sc[e], r[e], n[e]);
        c.store(ro, r);
        c.hat(r, a.layer, a.eps, inv_d, sum);
        if constexpr (!HOLD) {
            c.param(a.pre_gamma, 1.f, qg);
            c.param(a.pre_beta, 0.f, qb);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) r[e] = fmaf(r[e], qg[e], qb[e]);
        c.store(xo, r);
    }
}

template <int TPR, int VEC, int NV, typename TIO, typename TR> struct Fwd {
    static hipError_t run(const NormArgs &a, hipStream_t s) {
        const int rows = a.B * a.L, rpw = threads(TPR) / TPR;
        const int64_t need = (static_cast<int64_t>(rows) + rpw - 1) / rpw;
        const int grid = static_cast<int>(need < 2048 ? need : 2048);
        hipLaunchKernelGGL((block_norm_fwd<TPR, VEC, NV, TIO, TR>), dim3(grid), dim3(threads(TPR)), 0, s, a, rows);
        return hipGetLastError();
    }
};

}  // namespace

hipError_t launch_block_norm(const NormArgs &a, hipStream_t stream) {
    const bool out = aligned(a.resid_out, 16) && aligned(a.x, 16);
    return by_type<Fwd, 8, false>(a, a, out && vec_ok(a, 4), out && vec_ok(a, 8), stream);
}

}  // namespace ttt
