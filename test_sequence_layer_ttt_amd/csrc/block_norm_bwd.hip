// Gradients of the block norm (formulas of the forward in block_norm.hip).
//
// The backward reads the same rows and the two outputs' gradients, forms the
// forward's values again in registers (nothing is saved by the forward), and
// keeps the per-column sums of the parameters' gradients in registers over
// all rows of a workgroup; column_sums joins the workgroups in a fixed order.
//     g  = dr' + rstd_r (h - [mean h] - rhat mean(h rhat)),  h = dx pre_gamma
//     dresid = scale g,   dgate = g n act',   dn = g act
//     dy = rstd_y (k - [mean k] - yhat mean(k yhat)),        k = dn post_gamma
// ([..]: with the mean's removal only).
// B=4 L=2048 D=768 bf16: 101 MB in 30 us, 3.4 TB/s; bound by registers, which
// the columns' sums and two rows take: two waves a SIMD hide less of the loads
// and of four dependent row sums than the forward's do. Vector units are busy
// 61 % of the time (90 instructions a value), waves wait 46 % of theirs.
#include "block_norm.hpp"

namespace ttt {
namespace {

using namespace norm;

// column quantities of the backward's partials
enum { Q_POST_G, Q_PRE_G, Q_SCALE, Q_POST_B, Q_PRE_B, Q_GATE, Q_N };

// BETAS: the betas' column sums too
template <int TPR, int VEC, int NV, bool BETAS, typename TIO, typename TR>
__global__ __launch_bounds__(threads(TPR), VEC * NV <= 12 ? 2 : 1) void block_norm_bwd(NormBwdArgs ga) {
    typedef Cols<TPR, VEC, NV> C;
    constexpr int E = C::E, RPW = threads(TPR) / TPR;
    __shared__ float red[4][threads(TPR) / 64];
    __shared__ float comb[RPW > 1 ? RPW * TPR * E : 1];
    const NormArgs &a = ga.f;
    RowSum<TPR> sum{red};
    const C c{a.D, static_cast<int>(threadIdx.x % TPR)};
    const float inv_d = 1.0f / static_cast<float>(a.D);
    // rows of this workgroup: with a gate for each sequence those of sequence
    // blockIdx.y, else of the whole batch
    const int rows = a.gmode == TTT_GATE_SEQUENCE ? a.L : a.B * a.L;
    const int row0 = a.gmode == TTT_GATE_SEQUENCE ? blockIdx.y * a.L : 0;
    const int step = gridDim.x * RPW;
    float acc[Q_N][E] = {};  // BETAS false: two of them are never touched
    struct In {  // a row's inputs, fetched ahead
        typename C::template Raws<TR> resid, dro;
        typename C::template Raws<TIO> y, dx, gate;
        bool live;
    } next;
    auto fetch = [&](int i) {
        const int row = row0 + i, b = row / a.L, t = row - b * a.L;
        const int64_t at = static_cast<int64_t>(row) * a.D;
        next.live = !a.lens || t < a.lens[b];
        if (!next.live) return;
        c.fetch(static_cast<const TIO *>(a.y) + b * a.yb + t * a.yt, next.y);
        c.fetch(static_cast<const TR *>(a.resid) + b * a.rb + t * a.rt, next.resid);
        c.fetch(static_cast<const TIO *>(ga.dx) + at, next.dx);
        c.fetch(static_cast<const TR *>(ga.dresid_out) + at, next.dro);
        if (a.gmode == TTT_GATE_TOKEN) c.fetch(static_cast<const TIO *>(a.gate) + b * a.gb + t * a.gt, next.gate);
    };
    // where the sums leave registers for it
    constexpr bool AHEAD = E <= 8;
    int i = blockIdx.x * RPW + threadIdx.x / TPR;
    if (AHEAD && i < rows) fetch(i);
    for (; i < rows; i += step) {
        const int row = row0 + i;
        const int64_t at = static_cast<int64_t>(row) * a.D;
        if (!AHEAD) fetch(i);
        const In in = next;  // held as it is stored, unpacked where it is used
        if (AHEAD && i < rows - step) fetch(i + step);
        float u[E], v[E], w[E], yh[E], dxv[E];
        float ga_v[E], nd[E];  // the gate's value; what its derivative multiplies
        if (!in.live) {  // past the sequence's end: zeros, nothing read
#pragma unroll
            for (int e = 0; e < E; ++e) u[e] = 0.f;
            c.store(static_cast<TR *>(ga.dresid) + at, u);
            c.store(static_cast<TIO *>(ga.dy) + at, u);
            if (a.gmode == TTT_GATE_TOKEN) c.store(static_cast<TIO *>(ga.dgate) + at, u);
            continue;
        }
        auto gate = [&](float (&g)[E]) {
            if (a.gmode == TTT_GATE_TOKEN) c.unpack(in.gate, g);
            if (a.gmode == TTT_GATE_CHANNEL) c.load(static_cast<const float *>(a.gate), g);
            if (a.gmode == TTT_GATE_SEQUENCE) c.load(static_cast<const float *>(a.gate) + static_cast<int64_t>(row / a.L) * a.D, g);
        };
        c.unpack(in.y, yh);
        const float yr = c.hat(yh, a.layer, a.eps, inv_d, sum);
        // u: r', then its normalised value
        c.unpack(in.resid, w);
        c.param(a.scale, 1.f, u);
#pragma unroll
        for (int e = 0; e < E; ++e) u[e] *= w[e];
        c.param(a.post_gamma, 1.f, v);
        c.param(a.post_beta, 0.f, w);
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = fmaf(yh[e], v[e], w[e]);  // the norm after the block
        if (a.gmode != TTT_GATE_NONE) {
            gate(v);
            activate(a.act, v, ga_v, nd);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                u[e] = fmaf(ga_v[e], w[e], u[e]);
                nd[e] *= w[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) u[e] += w[e];
        }
        const float rr = c.hat(u, a.layer, a.eps, inv_d, sum);
        c.unpack(in.dx, dxv);
        c.param(a.pre_gamma, 1.f, v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            acc[Q_PRE_G][e] = fmaf(dxv[e], u[e], acc[Q_PRE_G][e]);
            if (BETAS) acc[Q_PRE_B][e] += dxv[e];
            dxv[e] *= v[e];
        }
        c.unhat(dxv, u, rr, a.layer, inv_d, sum);
        c.unpack(in.dro, v);  // dxv: the whole gradient of r'
#pragma unroll
        for (int e = 0; e < E; ++e) dxv[e] += v[e];
        c.unpack(in.resid, w);
        c.param(a.scale, 1.f, v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            acc[Q_SCALE][e] = fmaf(dxv[e], w[e], acc[Q_SCALE][e]);
            u[e] = dxv[e] * v[e];
        }
        c.store(static_cast<TR *>(ga.dresid) + at, u);
        c.param(a.post_gamma, 1.f, v);
        if (a.gmode != TTT_GATE_NONE) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                u[e] = dxv[e] * nd[e];
                dxv[e] *= ga_v[e];
            }
            if (a.gmode == TTT_GATE_TOKEN) {
                c.store(static_cast<TIO *>(ga.dgate) + at, u);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) acc[Q_GATE][e] += u[e];
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            acc[Q_POST_G][e] = fmaf(dxv[e], yh[e], acc[Q_POST_G][e]);
            if (BETAS) acc[Q_POST_B][e] += dxv[e];
            w[e] = dxv[e] * v[e];
        }
        c.unhat(w, yh, yr, a.layer, inv_d, sum);
        c.store(static_cast<TIO *>(ga.dy) + at, w);
    }
    float *part = ga.ws + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * Q_N * a.D;
    const bool want[Q_N] = {ga.dpost_gamma != nullptr, ga.dpre_gamma != nullptr, ga.dscale != nullptr,
                            ga.dpost_beta != nullptr, ga.dpre_beta != nullptr,
                            a.gmode == TTT_GATE_CHANNEL || a.gmode == TTT_GATE_SEQUENCE};
#pragma unroll
    for (int q = 0; q < Q_N; ++q) {
        if (!want[q] || (!BETAS && (q == Q_POST_B || q == Q_PRE_B))) continue;
        if constexpr (RPW > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e) comb[(e * RPW + threadIdx.x / TPR) * TPR + c.i] = acc[q][e];
            __syncthreads();
            if (threadIdx.x < TPR) {
                float s[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    s[e] = 0.f;
#pragma unroll
                    for (int k = 0; k < RPW; ++k) s[e] += comb[(e * RPW + k) * TPR + c.i];
                }
                c.store(part + static_cast<int64_t>(q) * a.D, s);
            }
        } else {
            c.store(part + static_cast<int64_t>(q) * a.D, acc[q]);
        }
    }
}

template <int TPR, int VEC, int NV, typename TIO, typename TR> struct Bwd {
    static hipError_t run(const NormBwdArgs &g, hipStream_t s) {
        const NormArgs &a = g.f;
        int64_t groups;
        int nq;
        block_norm_backward_partials(a.B, a.L, a.D, a.gmode, &groups, &nq);
        const int outer = a.gmode == TTT_GATE_SEQUENCE ? a.B : 1;
        const dim3 grid(static_cast<unsigned>(groups / outer), outer);
        if (g.dpost_beta || g.dpre_beta)
            hipLaunchKernelGGL((block_norm_bwd<TPR, VEC, NV, true, TIO, TR>), grid, dim3(threads(TPR)), 0, s, g);
        else
            hipLaunchKernelGGL((block_norm_bwd<TPR, VEC, NV, false, TIO, TR>), grid, dim3(threads(TPR)), 0, s, g);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        ColumnSums c{g.ws, static_cast<int64_t>(nq) * a.D, static_cast<int>(groups)};
        const int64_t D = a.D;
        c.add(Q_POST_G * D, a.D, 1, g.dpost_gamma);
        c.add(Q_PRE_G * D, a.D, 1, g.dpre_gamma);
        c.add(Q_SCALE * D, a.D, 1, g.dscale);
        c.add(Q_POST_B * D, a.D, 1, g.dpost_beta);
        c.add(Q_PRE_B * D, a.D, 1, g.dpre_beta);
        if (a.gmode == TTT_GATE_CHANNEL || a.gmode == TTT_GATE_SEQUENCE)
            c.add(Q_GATE * D, a.D, outer, static_cast<float *>(g.dgate));
        return launch_column_sums(c, s);
    }
};

}  // namespace

void block_norm_backward_partials(int B, int L, int D, int gmode, int64_t *groups, int *quantities) {
    const int rpw = D <= 1024 ? 4 : 1;  // rows a workgroup holds at a time
    const int64_t outer = gmode == TTT_GATE_SEQUENCE ? B : 1;
    const int64_t rows = gmode == TTT_GATE_SEQUENCE ? L : static_cast<int64_t>(B) * L;
    int64_t per = (rows + rpw - 1) / rpw;
    const int64_t most = outer < 512 ? 512 / outer : 1;
    if (per > most) per = most;
    if (per < 1) per = 1;
    *groups = outer * per > 0 ? outer * per : 1;
    *quantities = Q_N;
}

hipError_t launch_block_norm_backward(const NormBwdArgs &g, hipStream_t stream) {
    const bool out = aligned(g.dresid_out, 16) && aligned(g.dx, 16) && aligned(g.dresid, 16) &&
                     aligned(g.dy, 16) && aligned(g.dgate, 16) && aligned(g.ws, 16);
    const bool v = out && vec_ok(g.f, 4);
    return by_type<Bwd, 4, true>(g, g.f, v, v, stream);
}

}  // namespace ttt
