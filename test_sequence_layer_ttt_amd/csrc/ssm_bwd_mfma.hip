// The state space scan's gradients on the matrix cores: bf16 features, P <= 64,
// N <= 128. With the notation of ssm_mfma.hip, P_ij = exp(l_i - l_j),
// G_ij = C_i . B_j, E_ij = dy_i . x_j, S the state before a chunk and R the
// loss's gradient in the state behind it,
//     dC_i = sum_{j <= i} P_ij E_ij D_j B_j + exp(l_i) S dy_i
//     dB_j = D_j (sum_{i >= j} P_ij E_ij C_i + exp(l_63 - l_j) R x_j)
//     dx_j = D_j (sum_{i >= j} P_ij G_ij dy_i + exp(l_63 - l_j) B_j R) + D dy_j
// and what the decay's gradient is made of (ssm_bwd.hip), W_ij = P_ij G_ij E_ij D_j,
//     row_i = sum_{j < i} W_ij,   re_i = exp(l_i) C_i . (S dy_i)
//     col_j = sum_{i > j} W_ij,   co_j = D_j exp(l_63 - l_j) B_j . (R x_j)
// with the sums of W over the six pairs of different 16-token tiles.
//
// Two sweeps with one shape: forwards with S (own token i; rows X, B in LDS)
// and backwards with R (own token j; rows dY, C in LDS). A wave makes the
// outputs of its 16 tokens, transposed, as in ssm_mfma.hip; its own tokens'
// rows of the other pair (dY, C or x, B) are operand fragments straight from
// global memory, in the contraction order of the lanes' outputs, so they also
// serve the dot products with those outputs.
//  * The row and col sums are fp32: G and E are products of bf16 inputs summed
//    in fp32, and S dy (R x) takes the state in three bf16 parts. They feed
//    dA and ddt, where they are subtracted; dx, dB, dC are stored as bf16.
//    dx takes the decayed products and R as bf16 operands, dB and dC take
//    theirs in two bf16 parts (a group's heads add up their roundings).
//  * dB and dC of each head go out in fp32 and are summed over the group's
//    heads in a fixed order by ssm_bwd.hip.
// Bound by issue and latency of the many small products; two workgroups share
// a compute unit (N = 128: one, its LDS holds the state's three parts). 43 us
// for B=4 L=2048 H=12 N=64, both sweeps.
#include <type_traits>

#include "ssm_tile.hpp"

namespace ttt {
namespace {

using namespace ssm;

template <int N> struct BwdSmem {
    static constexpr int NS = N + 8;
    uint16_t v[2][Q * XS];      // [token][feature]: X or dY
    uint16_t k[2][Q * NS];      // [token][n]: B or C
    uint16_t s[3][64 * NS];     // the state's (gradient's) three parts, [feature][n]
    ChunkDecay d[2];
};

// what rounding to bf16 leaves
__device__ __forceinline__ f32x4 rest(f32x4 v) {
    const uint2 p = __builtin_bit_cast(uint2, pack4(v));
    return v - unpack4(p);
}
// place of the sum over rows of tile i and columns of tile j < i (see ssm.hpp)
__device__ __forceinline__ int pair_index(int i, int j) { return j == 0 ? i - 1 : j + i; }

struct SweepArgs {
    SsmBwdArgs g;
    SsmBwdWs w;
};

// a lane's part of row r in the order of its output rows: features 32 kb + 4 g
// .. + 3 and 32 kb + 16 + 4 g .. + 3
template <typename T>
__device__ __forceinline__ bf16x8 own_frag(const T *row, int kb, int g) {
    const uint2 a = *reinterpret_cast<const uint2 *>(row + 32 * kb + 4 * g);
    const uint2 b = *reinterpret_cast<const uint2 *>(row + 32 * kb + 16 + 4 * g);
    return __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
}
// the same from a row of `cols` in global memory
template <Fit FIT> __device__ __forceinline__ bf16x8 own_frag(const bf16_t *row, int kb, int g, int cols) {
    if constexpr (FIT == FULL) return own_frag(row, kb, g);
    if constexpr (FIT == WIDE) {
        const int f0 = 32 * kb + 4 * g, f1 = f0 + 16;
        const uint2 a = *reinterpret_cast<const uint2 *>(row + min(f0, cols - 4));
        const uint2 b = *reinterpret_cast<const uint2 *>(row + min(f1, cols - 4));
        return __builtin_bit_cast(bf16x8, make_uint4(f0 < cols ? a.x : 0u, f0 < cols ? a.y : 0u, f1 < cols ? b.x : 0u,
                                                     f1 < cols ? b.y : 0u));
    }
    const uint2 a = four(row, 32 * kb + 4 * g, cols), b = four(row, 32 * kb + 16 + 4 * g, cols);
    return __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
}
// values of output tile t (16 t + 4 g .. + 3) from such fragments
template <int KB> __device__ __forceinline__ f32x4 own_quad(const bf16x8 (&f)[KB], int t) {
    const uint4 r = __builtin_bit_cast(uint4, f[t / 2]);
    return t % 2 ? unpack4(make_uint2(r.z, r.w)) : unpack4(make_uint2(r.x, r.y));
}

template <int N, Fit FIT, bool REV>
__device__ __forceinline__ void sweep(const SweepArgs &w, BwdSmem<N> &sm) {
    constexpr int NS = BwdSmem<N>::NS, KB = N / 32, TN = N / 16;
    constexpr int NT = N >= 64 ? N / 64 : 1, UT = N >= 64 ? 4 : 2;  // the wave's part of the state
    const SsmBwdArgs &ga = w.g;
    const SsmArgs &a = ga.f;
    const int lane = threadIdx.x % 64, wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), g = lane / 16, c = lane % 16;
    int bs, h;
    place(blockIdx.x, a.B * a.nseg, a.H, bs, h);
    const int b = bs / a.nseg, seg = bs % a.nseg, gr = h / (a.H / a.G), bh = b * a.H + h;
    const int n = a.lens ? max(0, min(a.lens[b], a.L)) : a.L;
    const int64_t s0 = static_cast<int64_t>(seg) * a.seglen;
    const int t0 = static_cast<int>(s0 < a.L ? s0 : a.L);
    const int t1 = static_cast<int>(s0 + a.seglen < a.L ? s0 + a.seglen : a.L);
    const int te = max(t0, min(t1, n));
    const float Dh = a.D ? a.D[h] : 0.f;
    const float *prep = w.w.prep + static_cast<int64_t>(bh) * ((a.L + Q - 1) / Q) * 4 * Q;
    const SsmOperand &ov = REV ? ga.dy : a.x, &oz = REV ? a.x : ga.dy;
    const SsmOperand &ok = REV ? a.Cm : a.Bm, &oq = REV ? a.Bm : a.Cm;
    const bf16_t *vp = static_cast<const bf16_t *>(ov.p) + b * ov.sb + h * ov.sh;
    const bf16_t *zp = static_cast<const bf16_t *>(oz.p) + b * oz.sb + h * oz.sh;
    const bf16_t *kp = static_cast<const bf16_t *>(ok.p) + b * ok.sb + gr * ok.sh;
    const bf16_t *qp = static_cast<const bf16_t *>(oq.p) + b * oq.sb + gr * oq.sh;
    bf16_t *dxp = static_cast<bf16_t *>(const_cast<void *>(ga.dx.p)) + b * ga.dx.sb + h * ga.dx.sh;
    const int Nn = FIT == FULL ? N : a.N, P = FIT == FULL ? 64 : a.P;  // the tile's rest is zeros
    float *ph = (REV ? w.w.dBh : w.w.dCh) + static_cast<int64_t>(bh) * a.L * Nn;
    const int64_t tok0 = static_cast<int64_t>(bh) * a.L, inter = static_cast<int64_t>(a.B) * a.H * a.L;
    const int64_t tiles0 = static_cast<int64_t>(bh) * ((a.L + Q - 1) / Q);
    const int nt0 = N >= 64 ? NT * wv : wv % 2, u0 = N >= 64 ? 0 : 2 * (wv / 2);
    const int64_t NP = static_cast<int64_t>(Nn) * P;

    f32x4 st[NT][UT];
    const float *init = (REV ? w.w.sr : w.w.sf) + (static_cast<int64_t>(bh) * a.nseg + seg) * NP;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int u = 0; u < UT; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int k = 16 * (nt0 + i) + 4 * g + r, p = 16 * (u0 + u) + c;
                st[i][u][r] = FIT == FULL || (k < Nn && p < P) ? init[k * P + p] : 0.f;
            }

    Stage<64, FIT> sv;
    Stage<N, FIT> sk;
    bf16x8 zn[2], qn[KB];
    StageDecay sd;
    auto fetch_own = [&](int t) {
        const int64_t own = t + min(16 * wv + c, min(Q, te - t) - 1);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) zn[kb] = own_frag<FIT>(zp + own * oz.st, kb, g, P);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) qn[kb] = own_frag<FIT>(qp + own * oq.st, kb, g, Nn);
    };
    auto fetch = [&](int t) {
        const int count = min(Q, te - t);
        sv.fetch(vp + static_cast<int64_t>(t) * ov.st, ov.st, count, P);
        sk.fetch(kp + static_cast<int64_t>(t) * ok.st, ok.st, count, Nn);
        if (FIT != SINGLE) fetch_own(t);
        sd.fetch(prep + static_cast<int64_t>(t / Q) * 4 * Q);
    };
    auto put = [&](int t, int buf) {
        if (FIT == SINGLE) fetch_own(t);
        sv.put(sm.v[buf], XS, P);
        sk.put(sm.k[buf], NS, Nn);
        sd.put(sm.d[buf]);
    };
    auto share_state = [&]() {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int u = 0; u < UT; ++u) {
                uint2 p[3];
                split3(st[i][u][0], st[i][u][1], p[0].x, p[1].x, p[2].x);
                split3(st[i][u][2], st[i][u][3], p[0].y, p[1].y, p[2].y);
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    *reinterpret_cast<uint2 *>(&sm.s[k][(16 * (u0 + u) + c) * NS + 16 * (nt0 + i) + 4 * g]) = p[k];
            }
    };
    const int nc = (te - t0 + Q - 1) / Q;
    auto chunk = [&](int i) { return t0 + (REV ? nc - 1 - i : i) * Q; };
    if (nc) {
        fetch(chunk(0));
        put(chunk(0), 0);
        share_state();
    }
    for (int ci = 0; ci < nc; ++ci) {
        const int t = chunk(ci), buf = ci % 2;
        lds_barrier();
        bf16x8 z[2], q[KB];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) z[kb] = zn[kb];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) q[kb] = qn[kb];
        const bool more = ci + 1 < nc;
        if (more) fetch(chunk(ci + 1));
        const uint16_t *v = sm.v[buf], *kt = sm.k[buf];
        const ChunkDecay &d = sm.d[buf];
        const int o = 16 * wv + c;  // this lane's token
        const float hi = d.hi[o], lo = d.lo[o], step = d.step[o];
        const float reach = REV ? d.tail[o] : fast_exp2(hi);  // decay between the token and the state
        // products with the tokens before (behind) this lane's: rows m = 4 g + r
        float strict = 0.f, diag = 0.f, qs = 0.f, yx = 0.f;
        const bool live = t + o < te;
        bf16x8 vf[2][4];
        // straight-line code for each wave, tiles side by side, so that no product
        // waits at a branch or for the one before (51 -> 43 us)
        auto pairs = [&](auto wave) {
            constexpr int W = decltype(wave)::value;
            bf16x8 me[2][2], mg[2];
            float apart[4] = {};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                f32x4 pe[2], pg[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int mt = 2 * kb + k;
                    f32x4 G = {0.f, 0.f, 0.f, 0.f}, E = {0.f, 0.f, 0.f, 0.f};
                    if (REV ? mt >= W : mt <= W) {
#pragma unroll
                        for (int f = 0; f < KB; ++f) G = mfma32(own_frag(&kt[(16 * mt + c) * NS], f, g), q[f], G);
#pragma unroll
                        for (int f = 0; f < 2; ++f) E = mfma32(own_frag(&v[(16 * mt + c) * XS], f, g), z[f], E);
                        const int m = 16 * mt + 4 * g;
                        const f32x4 hm = *reinterpret_cast<const f32x4 *>(&d.hi[m]);
                        const f32x4 lm = *reinterpret_cast<const f32x4 *>(&d.lo[m]);
                        const f32x4 sm4 = *reinterpret_cast<const f32x4 *>(&d.step[m]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float l = (hm[r] - hi) + (lm[r] - lo);  // log2 P_{m,own} (REV), its negative else
                            float p = fast_exp2(REV ? l : -l);
                            if (!REV) p *= sm4[r];
                            const bool in = mt != W || (REV ? 4 * g + r >= c : 4 * g + r <= c), same = 4 * g + r == c;
                            const float e = in ? E[r] * p : 0.f;
                            const float ge = in ? G[r] * e : 0.f;
                            if (mt == W) {
                                strict += same ? 0.f : ge;
                                diag += same ? ge : 0.f;
                            } else {
                                apart[mt] += ge;
                            }
                            E[r] = e;
                            G[r] = in ? G[r] * p : 0.f;
                        }
                    }
                    pe[k] = E;
                    pg[k] = G;
                }
                me[kb][0] = pack8(pe[0], pe[1]);
                me[kb][1] = pack8(rest(pe[0]), rest(pe[1]));
                if constexpr (REV) mg[kb] = pack8(pg[0], pg[1]);
            }
            // a column's (row's) sum over the tiles, and the tiles' sums over the wave
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                strict += apart[mt];
                if (REV && mt > W) {
                    const float s = rows4_sum(row16_sum(apart[mt] * step));
                    if (lane == 0) w.w.tiles[(tiles0 + t / Q) * 8 + pair_index(mt, W)] = s;
                }
            }
            // over n: the state times z, its product with q, and the tokens' part
            f32x4 acc[TN];
#pragma unroll
            for (int tn = 0; tn < TN; ++tn) acc[tn] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int part = 2; part >= 0; --part)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int tn = 0; tn < TN; ++tn)
                        acc[tn] = mfma32(tokens_frag(sm.s[part], NS, kb, 16 * tn, g, c), z[kb], acc[tn]);
#pragma unroll
            for (int tn = 0; tn < TN; ++tn) {
                const f32x4 qv = own_quad(q, tn);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    qs = fmaf(qv[r], acc[tn][r], qs);
                    acc[tn][r] *= reach;
                }
            }
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                if (REV ? 2 * kb + 1 >= W : 2 * kb <= W) {
#pragma unroll
                    for (int tn = 0; tn < TN; ++tn) {
                        const bf16x8 f = tokens_frag(kt, NS, kb, 16 * tn, g, c);
                        acc[tn] = mfma32(f, me[kb][1], acc[tn]);
                        acc[tn] = mfma32(f, me[kb][0], acc[tn]);
                    }
                }
            }
            if (REV) {
#pragma unroll
                for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[tn][r] *= step;
            }
            if (live) {
#pragma unroll
                for (int tn = 0; tn < TN; ++tn) {
                    float *out = ph + static_cast<int64_t>(t + o) * Nn + 16 * tn + 4 * g;
                    if constexpr (FIT != SINGLE) {
                        if (FIT == FULL || 16 * tn + 4 * g < Nn) *reinterpret_cast<f32x4 *>(out) = acc[tn];
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (16 * tn + 4 * g + r < Nn) out[r] = acc[tn][r];
                    }
                }
            }
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int u = 0; u < 4; ++u) vf[kb][u] = tokens_frag(v, XS, kb, 16 * u, g, c);
            if constexpr (REV) {
                float out[4][4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int f = 0; f < KB; ++f) acc = mfma32(own_frag(&sm.s[0][(16 * u + c) * NS], f, g), q[f], acc);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[r] *= reach;
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb) {
                        if (2 * kb + 1 >= W) acc = mfma32(vf[kb][u], mg[kb], acc);
                    }
                    const f32x4 xv = own_quad(z, u);
                    float dyv[4];
                    vec_load<bf16_t, 4>(&v[o * XS + 16 * u + 4 * g], dyv);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        yx = fmaf(xv[r], dyv[r], yx);
                        out[u][r] = fmaf(step, acc[r], Dh * dyv[r]);
                    }
                }
                store_row<FIT>(dxp + static_cast<int64_t>(t + o) * ga.dx.st, live, out, g, P);
                yx = rows4_sum(yx);
            }
        };
        if (wv == 0) pairs(std::integral_constant<int, 0>());
        else if (wv == 1) pairs(std::integral_constant<int, 1>());
        else if (wv == 2) pairs(std::integral_constant<int, 2>());
        else pairs(std::integral_constant<int, 3>());
        strict = rows4_sum(strict);
        diag = rows4_sum(diag);
        qs = reach * rows4_sum(qs);
        if (live && g == 0) {
            const int64_t tok = tok0 + t + o;
            if constexpr (REV) {
                w.w.col[tok] = step * strict;
                w.w.col[inter + tok] = step * qs;
                w.w.xdu[tok] = strict + diag + qs;
                w.w.dyx[tok] = yx;
            } else {
                w.w.row[tok] = strict;
                w.w.row[inter + tok] = qs;
            }
        }
        if (more) {  // the state before the next chunk
            const float whole = fast_exp2(d.total());
            // the chunk's share is summed by itself, as those at the segments' borders are
            f32x4 share[NT][UT] = {};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const int j0 = 32 * kb + 4 * g, j1 = j0 + 16;
                f32x4 w0 = *reinterpret_cast<const f32x4 *>(REV ? &d.hi[j0] : &d.tail[j0]);
                f32x4 w1 = *reinterpret_cast<const f32x4 *>(REV ? &d.hi[j1] : &d.tail[j1]);
                const f32x4 p0 = *reinterpret_cast<const f32x4 *>(&d.step[j0]);
                const f32x4 p1 = *reinterpret_cast<const f32x4 *>(&d.step[j1]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    w0[r] = REV ? fast_exp2(w0[r]) : w0[r] * p0[r];
                    w1[r] = REV ? fast_exp2(w1[r]) : w1[r] * p1[r];
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    bf16x8 kw[3];
                    weigh<3>(tokens_frag(kt, NS, kb, 16 * (nt0 + i), g, c), w0, w1, kw);
#pragma unroll
                    for (int k = 2; k >= 0; --k)
#pragma unroll
                        for (int u = 0; u < UT; ++u)
                            share[i][u] = mfma32(kw[k], N >= 64 || wv < 2 ? vf[kb][u] : vf[kb][2 + u % 2], share[i][u]);
                }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int u = 0; u < UT; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) st[i][u][r] = fmaf(st[i][u][r], whole, share[i][u][r]);
            put(chunk(ci + 1), buf ^ 1);
            lds_barrier();  // every wave has read the state's parts
            share_state();
        }
    }
    // rows past the sequence's end are zeros
    const float zero[4] = {};
    for (int t = te + static_cast<int>(threadIdx.x) / 16; t < t1; t += 16) {
        const int e = threadIdx.x % 16;
        for (int k = e; k < Nn; k += 16) ph[static_cast<int64_t>(t) * Nn + k] = 0.f;
        if constexpr (REV) store4<FIT>(dxp + static_cast<int64_t>(t) * ga.dx.st, 4 * e, P, zero);
    }
}

// blockIdx.y: the sweep backwards (the longer one) first
template <int N, Fit FIT> __global__ __launch_bounds__(256, N == 128 ? 1 : 2) void sweeps(SweepArgs w) {
    __shared__ BwdSmem<N> sm;
    if (blockIdx.y == 0)
        sweep<N, FIT, true>(w, sm);
    else
        sweep<N, FIT, false>(w, sm);
}

template <Fit FIT> hipError_t run(const SweepArgs &w, hipStream_t s) {
    const SsmArgs &a = w.g.f;
    const dim3 grid(static_cast<unsigned>(a.B) * a.H * a.nseg, 2);
    if (a.N <= 32)
        hipLaunchKernelGGL((sweeps<32, FIT>), grid, dim3(256), 0, s, w);
    else if (a.N <= 64)
        hipLaunchKernelGGL((sweeps<64, FIT>), grid, dim3(256), 0, s, w);
    else
        hipLaunchKernelGGL((sweeps<128, FIT>), grid, dim3(256), 0, s, w);
    return hipGetLastError();
}

}  // namespace

bool ssm_bwd_mfma_supported(const SsmBwdArgs &g) { return ssm_mfma_supported(g.f); }

hipError_t launch_ssm_bwd_mfma(const SsmBwdArgs &g, hipStream_t stream) {
    const SsmArgs &a = g.f;
    const int NP = a.N * a.P;
    const SsmBwdWs s = ssm_backward_ws(a);
    hipError_t e;
    if ((e = launch_ssm_prep(a, s.prep, stream)) != hipSuccess) return e;
    if ((e = launch_ssm_shares_mfma(a, g.dy, s.prep, s.sf, s.sr, s.decay, stream)) != hipSuccess) return e;
    const SsmCarry cf{a.state, s.decay, s.sf, s.last, 0}, cr{g.dstate_out, s.decay, s.sr, g.dstate, 1};
    if ((e = launch_ssm_carry(a.B * a.H, NP, a.nseg, cf, &cr, stream)) != hipSuccess) return e;
    const SweepArgs w{g, s};
    const int fit = ssm_fit(a, g.dy, g.dx);
    e = fit == FULL ? run<FULL>(w, stream) : fit == WIDE ? run<WIDE>(w, stream) : run<SINGLE>(w, stream);
    if (e != hipSuccess) return e;
    return launch_ssm_bwd_finish(g, true, stream);
}

}  // namespace ttt
