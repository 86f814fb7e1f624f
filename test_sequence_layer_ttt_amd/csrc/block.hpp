// Internal launchers (host side) of the operators around the layer: the short
// causal convolution, the selective state space scan and the block norm.
// Arguments are validated by the C ABI before these are called; each enqueues
// on `stream` and returns the launch status. All strides are in elements; the
// innermost dimension is contiguous.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ttt {

struct ConvArgs {
    int B, L, C, K, io, silu;
    const void *x;
    int64_t xb, xt;        // batch and token strides of x
    const float *w, *bias;  // [C,K], [C] or null
    const void *state;     // [B,K-1,C] or null (zeros)
    const int *lens;       // [B] or null
    void *y;               // forward: [B,L,C]
    int64_t yb, yt;
    void *state_out;       // forward: [B,K-1,C] or null
};

struct ConvBwdArgs {
    ConvArgs f;  // forward arguments (y, state_out unused)
    const void *dy;
    int64_t dyb, dyt;
    const void *dstate_out;  // [B,K-1,C] or null
    void *dx;
    int64_t dxb, dxt;
    float *dw, *dbias;  // dbias null if bias is
    void *dstate;       // [B,K-1,C], null if state is
    float *ws;          // conv_backward_blocks(...) * C * (K + 1) floats
};

hipError_t launch_conv_forward(const ConvArgs &a, hipStream_t stream);
hipError_t launch_conv_step(const ConvArgs &a, hipStream_t stream);  // state read and written
int64_t conv_backward_blocks(int B, int L, int C);
hipError_t launch_conv_backward(const ConvBwdArgs &a, hipStream_t stream);

struct NormArgs {
    int B, L, D, io, rio, layer;  // io: y, gate per token, x; rio: resid
    int act, gmode;               // TTT_ACT_*, TTT_GATE_*
    float eps;
    const void *resid;
    int64_t rb, rt;
    const void *y;
    int64_t yb, yt;
    const void *gate;  // [D], [B,D] fp32 or [B,L,D] io
    int64_t gb, gt;
    const float *post_gamma, *post_beta, *pre_gamma, *pre_beta, *scale;  // [D] or null
    const int *lens;
    void *resid_out, *x;  // [B,L,D]
};

struct NormBwdArgs {
    NormArgs f;  // forward arguments (resid_out, x unused)
    const void *dresid_out, *dx;  // [B,L,D]
    void *dresid, *dy, *dgate;    // [B,L,D]; dgate as gate
    float *dpost_gamma, *dpost_beta, *dpre_gamma, *dpre_beta, *dscale;
    float *ws;
};

hipError_t launch_block_norm(const NormArgs &a, hipStream_t stream);
// workgroups and column quantities of the backward's partial sums [groups][quantities][D]
void block_norm_backward_partials(int B, int L, int D, int gmode, int64_t *groups, int *quantities);
hipError_t launch_block_norm_backward(const NormBwdArgs &a, hipStream_t stream);

// Sums over the rows of part[rows][stride], for up to 8 ranges of columns:
// out[o * cols + c] = sum of part[r][off + c] over the o-th of `outer` equal
// runs of rows, in a fixed order.
struct ColumnSums {
    const float *part;
    int64_t stride;
    int rows;
    int n = 0;
    struct Range {
        int64_t off;
        int cols, outer;
        float *out;
    } q[8] = {};
    void add(int64_t off, int cols, int outer, float *out) {
        if (out) q[n++] = Range{off, cols, outer, out};
    }
};
hipError_t launch_column_sums(const ColumnSums &c, hipStream_t stream);

}  // namespace ttt
