// Internal interface of the selective state space scan (see ttt.h for the
// formulas). A sequence is cut into segments; each segment's own contribution
// to the state is formed for all segments at once, carried over the segments
// in order, and the outputs are then formed for all segments at once from the
// states at their borders.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ttt {

// A per-token, per-head operand: element (b, t, h, i) at p + b*sb + t*st + h*sh + i.
// `shared`: h counts groups of heads.
struct SsmOperand {
    const void *p;
    int64_t sb, st, sh;
};

struct SsmArgs {
    int B, L, H, P, G, N, io;
    SsmOperand x, dt, Bm, Cm;  // dt has no innermost dimension
    const float *A, *D, *dt_bias;  // [H]; D, dt_bias may be null
    const float *state;            // [B,H,N,P] or null
    const int *lens;
    SsmOperand y;
    float *state_out;  // [B,H,N,P] or null
    float *ws;
    int nseg, seglen;
};

struct SsmBwdArgs {
    SsmArgs f;
    SsmOperand dy;
    const float *dstate_out;  // [B,H,N,P] or null
    SsmOperand dx, ddt, dB, dC;
    float *dA, *dD, *ddt_bias, *dstate;  // dD, ddt_bias, dstate may be null
};

// segments of the forward and of the backward
void ssm_segments(int B, int L, int H, int N, bool mfma, bool backward, int *nseg, int *seglen);
bool ssm_mfma_supported(const SsmArgs &a);
// how x, B, C, p and q lie in the MFMA kernels' tiles (ssm_tile.hpp, Fit)
int ssm_fit(const SsmArgs &a, const SsmOperand &p, const SsmOperand &q);
// Values (of VD features) that a lane of the walks holds, 16 lanes side by side:
// their blocks are of 16 times as many.
int ssm_lane_values(int B, int L, int H, int VD);
// workspace floats
size_t ssm_forward_floats(int B, int L, int H, int P, int N, int nseg);
size_t ssm_backward_floats(int B, int L, int H, int P, int N, int nseg);

hipError_t launch_ssm_step(const SsmArgs &a, hipStream_t stream);  // L = 1, state_out in place
hipError_t launch_ssm_forward(const SsmArgs &a, hipStream_t stream);
hipError_t launch_ssm_backward(const SsmBwdArgs &a, hipStream_t stream);

// Parts of the launches above.
//
// The carry over segments, forward: S[0] = first (or zeros), S[s+1] = decay[s]
// S[s] + share[s]; on entry seg holds the shares [B,H,nseg,N,P], on return the
// state before each segment. Reverse: S[nseg] = first, S[s] = decay[s] S[s+1] +
// share[s]; on return seg[s] = S[s+1], the state's gradient behind segment s.
// `out` (or null) receives what the walk ends with. One or two in a launch.
struct SsmCarry {
    const float *first, *decay;
    float *seg, *out;
    int reverse;
};
hipError_t launch_ssm_carry(int BH, int NP, int nseg, const SsmCarry &c, const SsmCarry *other, hipStream_t stream);

// What the backward's second half needs (ssm_bwd.hip).
struct SsmBwdWs {
    float *sf, *sr;   // [B,H,nseg,N,P] states before, gradients behind each segment
    float *last;      // [B,H,N,P] state after the last segment
    float *decay;     // [B,H,nseg]
    float *dBh, *dCh; // [B,H,L,N] per head
    // [blocks,B,H,L] per token. From the walks: the blocks of values' shares of
    // the strict products (row: of N, col: of P). From the sweeps: the part
    // within the 64-token chunk, then the part through the state before
    // (behind) it.
    float *row, *col;
    float *xdu, *dyx;  // x . du and dy . x, by blocks of P (sweeps: the first)
    int rows, cols;    // blocks of the walks
    float *tiles;      // [B,H,ceil(L/64),8] sweeps: sums over pairs of 16-token tiles (i, j),
                       // (1,0) (2,0) (3,0) (2,1) (3,1) (3,2)
    float *part;       // [B*nseg][3][H]
    float *prep;       // ssm_prep's chunks
    size_t floats;     // of all of them
};
SsmBwdWs ssm_backward_ws(const SsmArgs &a);
hipError_t launch_ssm_bwd_finish(const SsmBwdArgs &g, bool sweeps, hipStream_t stream);

hipError_t launch_ssm_states_valu(const SsmArgs &a, const SsmOperand *dy, float *seg, float *decay,
                                  hipStream_t stream);
hipError_t launch_ssm_mfma(const SsmArgs &a, hipStream_t stream);
// the segments' shares of the states and of their gradients, one launch
hipError_t launch_ssm_shares_mfma(const SsmArgs &a, const SsmOperand &dy, const float *prep, float *sf, float *sr,
                                  float *decay, hipStream_t stream);
// the chunks' decays for the MFMA kernels
size_t ssm_prep_floats(int B, int L, int H);
hipError_t launch_ssm_prep(const SsmArgs &a, float *out, hipStream_t stream);
bool ssm_bwd_mfma_supported(const SsmBwdArgs &g);
hipError_t launch_ssm_bwd_mfma(const SsmBwdArgs &g, hipStream_t stream);

}  // namespace ttt
