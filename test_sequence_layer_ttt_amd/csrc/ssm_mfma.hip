// The selective state space scan on the matrix cores: bf16 features, P <= 64,
// N <= 128 in tiles of 64 x 32, 64 or 128 (formulas in ttt.h). A workgroup of four waves walks over
// the 64-token chunks of one head's segment. With l_i the sum of D_t A over
// the chunk's tokens up to i and S the state before the chunk, a chunk is
//     M_ij = (C_i . B_j) exp(l_i - l_j) D_j  for j <= i, else 0
//     Y = M X + diag(exp(l)) C S + D X
//     S <- exp(l_63) S + (B diag(exp(l_63 - l) D))^T X.
//  * Wave w makes the outputs of tokens 16 w .. + 15, all transposed: B C^T
//    gives M^T with four tokens j of one i in a lane, which is the operand of
//    X^T M^T as it stands (no trip through LDS); Y^T gives four adjacent
//    features of one token to a lane.
//  * The state lives in accumulators, fp32: wave w holds N / 4 of its rows
//    (N = 32: half of the columns of 16). Where it goes on to the caller or to
//    another segment, its update takes X exactly as it is and B D exp(..) split
//    into three bf16 parts, so it is that of fp32 arithmetic; where it only
//    feeds C S of its own segment, one rounded part. Its copy for C S, in LDS,
//    is rounded to bf16, as is M: y is off by 1.9e-3 of its norm, of which
//    the rounding of y itself is 1.7e-3.
//  * X and B of the next chunk are fetched to registers while this one is
//    worked on, C straight to the fragment that needs it; X^T and B^T are read
//    from the row-major tiles by transposing LDS reads.
//  * A masked M_ij is a zero, and zero times an infinity is not. So infinities
//    and NaN of x do not enter the tiles: the waves that stage x put zeros there
//    and note each such feature's first token, from which on its outputs are
//    NaN, and its state. (B's only meet their own token's column of M, which is
//    selected.) Testing costs 1.5 us of the 8k prompt's 75.
//  * Few heads: the sequence is cut into segments that run side by side. A
//    first launch of the same walk without outputs gives each segment's share
//    of the state, carried over the segments by ssm_carry.
// Floor: x, y once (2 * 128 bytes a token and head), B and C from the L2 that
// the heads of a segment share; about 8 N * 64 + 4 * 64 * (N + 64) flops a
// token and head.
// Measured, bf16, P = 64: B=2 L=8192 H=32 N=64 outputs 43 us, shares 27 us (12
// segments; x and y once would be 28 us); L=32768 H=32 N=128 outputs 129 us,
// shares 90 us. Bound by latency and issue together: three workgroups (two at
// N = 128) of four waves a compute unit, 344 vector instructions for a wave and
// chunk, which hold the vector unit 55 % of the time, waves waiting 39 % of
// theirs. With 311 of them (no test of x) the first took 41 us; 35 without its
// stores, 39 without its loads. Straight-line code for each wave's tiles, D x as a product of its own and
// tiles without bank conflicts changed nothing (41 .. 42 us).
#include "ssm_tile.hpp"

namespace ttt {
namespace {

using namespace ssm;

template <int N, bool OUT> struct Smem {
    static constexpr int NS = N + 8;
    uint16_t x[2][Q * XS];   // [token][feature]
    uint16_t b[2][Q * NS];   // [token][n]
    uint16_t s[OUT ? 64 * NS : 8];  // the state's bf16 copy, [feature][n]
    ChunkDecay d[2];
    alignas(16) float f[OUT ? 4 : 1][Q];  // each wave's decays to its tokens' tile
    // features of x that are not finite, by the waves that found them: whether
    // there are any, and the first token where one is
    alignas(16) uint32_t found[OUT ? 2 : 1][4];
    int first[OUT ? 2 : 1][4][64];
};

struct MfmaArgs {
    SsmArgs a;
    const float *init;    // [B,H,(nseg,)N,P]
    int64_t init_stride;  // as in WalkArgs
    float *fin, *decay;   // decay: of each segment, from the shares forwards
    const float *prep;    // ssm_prep's chunks
};

// OUT: outputs and the state's update. Otherwise the segment's share of the
// state alone, or (REV) of the state's gradient: a walk from the segment's end
// over S <- exp(l_63) S + (C diag(exp(l)))^T dY, with C in Bm and dY in x.
template <int N, Fit FIT, bool OUT, bool REV, int PARTS>
__device__ __forceinline__ void chunks(const MfmaArgs &w, Smem<N, OUT> &sm) {
    constexpr int NS = Smem<N, OUT>::NS, KB = N / 32;
    constexpr int NT = N >= 64 ? N / 64 : 1;  // row tiles of the state in a wave
    constexpr int UT = N >= 64 ? 4 : 2;       // its feature tiles
    static_assert(!(OUT && REV), "outputs are made forwards");
    const SsmArgs &a = w.a;
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
    const float *prep = w.prep + static_cast<int64_t>(bh) * ((a.L + Q - 1) / Q) * 4 * Q;
    const bf16_t *xp = static_cast<const bf16_t *>(a.x.p) + b * a.x.sb + h * a.x.sh;
    const bf16_t *bp = static_cast<const bf16_t *>(a.Bm.p) + b * a.Bm.sb + gr * a.Bm.sh;
    const bf16_t *cp = static_cast<const bf16_t *>(a.Cm.p) + b * a.Cm.sb + gr * a.Cm.sh;
    bf16_t *yp = static_cast<bf16_t *>(const_cast<void *>(a.y.p)) + b * a.y.sb + h * a.y.sh;
    const int nt0 = N >= 64 ? NT * wv : wv % 2, u0 = N >= 64 ? 0 : 2 * (wv / 2);
    const int Nn = FIT == FULL ? N : a.N, P = FIT == FULL ? 64 : a.P;  // the tile's rest is zeros
    const int64_t NP = static_cast<int64_t>(Nn) * P;

    f32x4 st[NT][UT];
    const float *init = w.init ? w.init + (w.init_stride ? (static_cast<int64_t>(bh) * a.nseg + seg) * NP : bh * NP) : nullptr;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int u = 0; u < UT; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r)
            {
                const int k = 16 * (nt0 + i) + 4 * g + r, p = 16 * (u0 + u) + c;
                st[i][u][r] = init && (FIT == FULL || (k < Nn && p < P)) ? init[k * P + p] : 0.f;
            }

    Stage<64, FIT> sx;
    Stage<N, FIT> sb;
    bf16x8 cf[KB], cn[KB];
    StageDecay sd;
    auto fetch_own = [&](int t) {
        if constexpr (OUT) {
            const bf16_t *p = cp + static_cast<int64_t>(t + min(16 * wv + c, min(Q, te - t) - 1)) * a.Cm.st;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) cn[kb] = __builtin_bit_cast(bf16x8, eight<FIT>(p, 32 * kb + 8 * g, Nn));
        }
    };
    auto fetch = [&](int t) {  // the chunk at token t < te
        const int count = min(Q, te - t);
        sx.fetch(xp + static_cast<int64_t>(t) * a.x.st, a.x.st, count, P);
        sb.fetch(bp + static_cast<int64_t>(t) * a.Bm.st, a.Bm.st, count, Nn);
        if (FIT != SINGLE) fetch_own(t);
        sd.fetch(prep + static_cast<int64_t>(t / Q) * 4 * Q);
    };
    uint32_t marked = 0;  // what `found` says of this wave's buffers
    if constexpr (OUT) sm.found[0][wv] = sm.found[1][wv] = 0;
    auto put = [&](int t, int buf) {
        if (FIT == SINGLE) fetch_own(t);
        if constexpr (OUT) {
            const bool found = sx.put_finite(sm.x[buf], XS, P, sm.first[buf][wv]);
            if (found != (marked >> buf & 1)) {  // it holds what it held
                sm.found[buf][wv] = found;
                marked ^= 1u << buf;
            }
        } else {
            sx.put(sm.x[buf], XS, P);
        }
        sb.put(sm.b[buf], NS, Nn);
        sd.put(sm.d[buf]);
    };
    auto share_state = [&]() {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int u = 0; u < UT; ++u)
                *reinterpret_cast<s16x4 *>(&sm.s[(16 * (u0 + u) + c) * NS + 16 * (nt0 + i) + 4 * g]) = pack4(st[i][u]);
    };
    float total = 0.f;
    const int nc = (te - t0 + Q - 1) / Q;
    auto chunk = [&](int i) { return t0 + (REV ? nc - 1 - i : i) * Q; };
    if (nc) {
        fetch(chunk(0));
        put(chunk(0), 0);
        if constexpr (OUT) share_state();
    }
    for (int ci = 0; ci < nc; ++ci) {
        const int t = chunk(ci), buf = ci % 2;
        lds_barrier();
        if constexpr (OUT) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) cf[kb] = cn[kb];
        }
        const bool more = ci + 1 < nc;
        if (more) fetch(chunk(ci + 1));
        const uint16_t *x = sm.x[buf], *bt = sm.b[buf];
        const ChunkDecay &d = sm.d[buf];
        bool spoilt = false;
        if constexpr (OUT) {
            const uint4 q = *reinterpret_cast<const uint4 *>(sm.found[buf]);
            spoilt = __builtin_amdgcn_readfirstlane(q.x | q.y | q.z | q.w);
        }
        auto first = [&](int p) {  // the first token at which feature p is not finite
            int f = Q;
            for (int k = 0; k < 4; ++k)
                if (sm.found[buf][k]) f = min(f, sm.first[buf][k][p]);
            return f;
        };
        bf16x8 xf[2][4];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int u = 0; u < 4; ++u) xf[kb][u] = tokens_frag(x, XS, kb, 16 * u, g, c);
        if constexpr (OUT) {
            const int i = 16 * wv + c;  // this lane's token
            const float hi = d.hi[i];
            // decay from a token j of an earlier tile to the end of the tile
            // before this wave's, times D_j (one exp a lane), and from there
            // to token i: with A < 0 neither is above 1
            const float edge = wv ? d.hi[16 * wv - 1] : 0.f;
            sm.f[wv][lane] = lane < 16 * wv ? fast_exp2(edge - d.hi[lane]) * d.step[lane] : 0.f;
            const float ef = fast_exp2(hi - edge);
            bf16x8 mf[2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                f32x4 m[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int jt = 2 * kb + k;
                    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
                    if (jt <= wv) {
#pragma unroll
                        for (int q = 0; q < KB; ++q)
                            acc = mfma32(read16(&bt[(16 * jt + c) * NS + 32 * q + 8 * g]), cf[q], acc);
                        const int j = 16 * jt + 4 * g;
                        if (jt < wv) {
                            const f32x4 fj = *reinterpret_cast<const f32x4 *>(&sm.f[wv][j]);
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[r] *= fj[r] * ef;
                        } else {
                            const f32x4 hj = *reinterpret_cast<const f32x4 *>(&d.hi[j]);
                            const f32x4 sj = *reinterpret_cast<const f32x4 *>(&d.step[j]);
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                acc[r] = j + r <= i ? acc[r] * (fast_exp2(hi - hj[r]) * sj[r]) : 0.f;
                        }
                    }
                    m[k] = acc;
                }
                mf[kb] = pack8(m[0], m[1]);
            }
            f32x4 y[4];
            const float ei = fast_exp2(hi);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                y[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < KB; ++q) y[u] = mfma32(read16(&sm.s[(16 * u + c) * NS + 32 * q + 8 * g]), cf[q], y[u]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) y[u][r] *= ei;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                if (2 * kb <= wv) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) y[u] = mfma32(xf[kb][u], mf[kb], y[u]);
                }
            }
            float o[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float xv[4];
                vec_load<bf16_t, 4>(&x[i * XS + 16 * u + 4 * g], xv);
#pragma unroll
                for (int r = 0; r < 4; ++r) o[u][r] = fmaf(Dh, xv[r], y[u][r]);
            }
            if (__builtin_expect(spoilt, 0)) {
                for (int u = 0; u < 4; ++u)
                    for (int r = 0; r < 4; ++r)
                        if (i >= first(16 * u + 4 * g + r)) o[u][r] = NAN;
            }
            store_row<FIT>(yp + static_cast<int64_t>(t + i) * a.y.st, t + i < te, o, g, P);
        }
        const float whole = fast_exp2(d.total());
        total += d.total();
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int u = 0; u < UT; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) st[i][u][r] *= whole;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const int j0 = 32 * kb + 4 * g, j1 = j0 + 16;
            f32x4 w0, w1;
            if constexpr (REV) {
                w0 = *reinterpret_cast<const f32x4 *>(&d.hi[j0]);
                w1 = *reinterpret_cast<const f32x4 *>(&d.hi[j1]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    w0[r] = fast_exp2(w0[r]);
                    w1[r] = fast_exp2(w1[r]);
                }
            } else {
                w0 = *reinterpret_cast<const f32x4 *>(&d.tail[j0]);
                w1 = *reinterpret_cast<const f32x4 *>(&d.tail[j1]);
                const f32x4 p0 = *reinterpret_cast<const f32x4 *>(&d.step[j0]), p1 = *reinterpret_cast<const f32x4 *>(&d.step[j1]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    w0[r] *= p0[r];
                    w1[r] *= p1[r];
                }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                bf16x8 bw[PARTS];
                weigh<PARTS>(tokens_frag(bt, NS, kb, 16 * (nt0 + i), g, c), w0, w1, bw);
                // the smallest part first: the state off 9.6e-8, 1.15e-7 the other way
#pragma unroll
                for (int k = PARTS - 1; k >= 0; --k)
#pragma unroll
                    for (int u = 0; u < UT; ++u)
                        st[i][u] = mfma32(bw[k], N >= 64 || wv < 2 ? xf[kb][u] : xf[kb][2 + u % 2], st[i][u]);
            }
        }
        if (OUT && __builtin_expect(spoilt, 0)) {
            for (int u = 0; u < UT; ++u)
                if (first(16 * (u0 + u) + c) < Q)
                    for (int i = 0; i < NT; ++i)
                        for (int r = 0; r < 4; ++r) st[i][u][r] = NAN;
        }
        if (more) put(chunk(ci + 1), buf ^ 1);
        if constexpr (OUT) {
            if (more) {
                lds_barrier();  // every wave has read the state's copy
                share_state();
            }
        }
    }
    if constexpr (OUT) {  // rows past the sequence's end are zeros
        const float zero[4] = {};
        for (int t = te + threadIdx.x / 16; t < t1; t += 16)
            store4<FIT>(yp + static_cast<int64_t>(t) * a.y.st, threadIdx.x % 16 * 4, P, zero);
    }
    if (w.fin) {
        float *f = w.fin + (static_cast<int64_t>(bh) * (OUT ? 1 : a.nseg) + (OUT ? 0 : seg)) * NP;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int u = 0; u < UT; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int k = 16 * (nt0 + i) + 4 * g + r, p = 16 * (u0 + u) + c;
                    if (FIT == FULL || (k < Nn && p < P)) f[k * P + p] = st[i][u][r];
                }
    }
    // by the walk forwards alone: the one from the end adds the chunks up in another
    // order, which rounds differently, and runs at the same time
    if (!OUT && !REV && threadIdx.x == 0) w.decay[static_cast<int64_t>(bh) * a.nseg + seg] = exp2f(total);
}

// PARTS 3: the state goes on to the caller. 1: it does not (its exact value
// comes from the shares) and only feeds the outputs, through a bf16 copy.
template <int N, Fit FIT, int PARTS>
__global__ __launch_bounds__(256, N == 128 ? 2 : 3) void outputs(MfmaArgs w) {
    __shared__ Smem<N, true> sm;
    chunks<N, FIT, true, false, PARTS>(w, sm);
}
// blockIdx.y: the states' shares, then those of their gradients
template <int N, Fit FIT>
__global__ __launch_bounds__(256, N == 128 ? 2 : 3) void shares(MfmaArgs f, MfmaArgs r) {
    __shared__ Smem<N, false> sm;
    if (blockIdx.y == 0)
        chunks<N, FIT, false, false, 3>(f, sm);
    else
        chunks<N, FIT, false, true, 3>(r, sm);
}

template <int N, Fit FIT> hipError_t run(const MfmaArgs *out, const MfmaArgs *f, const MfmaArgs *r, hipStream_t s) {
    const SsmArgs &a = out ? out->a : f->a;
    const unsigned blocks = static_cast<unsigned>(a.B) * a.H * a.nseg;
    if (out && out->fin)
        hipLaunchKernelGGL((outputs<N, FIT, 3>), dim3(blocks), dim3(256), 0, s, *out);
    else if (out)
        hipLaunchKernelGGL((outputs<N, FIT, 1>), dim3(blocks), dim3(256), 0, s, *out);
    else
        hipLaunchKernelGGL((shares<N, FIT>), dim3(blocks, r ? 2 : 1), dim3(256), 0, s, *f, r ? *r : *f);
    return hipGetLastError();
}
template <Fit FIT> hipError_t run(const MfmaArgs *out, const MfmaArgs *f, const MfmaArgs *r, hipStream_t s) {
    const int N = out ? out->a.N : f->a.N;
    return N <= 32 ? run<32, FIT>(out, f, r, s) : N <= 64 ? run<64, FIT>(out, f, r, s) : run<128, FIT>(out, f, r, s);
}

hipError_t run(int fit, const MfmaArgs *out, const MfmaArgs *f, const MfmaArgs *r, hipStream_t s) {
    return fit == FULL ? run<FULL>(out, f, r, s) : fit == WIDE ? run<WIDE>(out, f, r, s) : run<SINGLE>(out, f, r, s);
}

bool wide(const SsmOperand &o) {  // rows of 16-byte accesses
    return (reinterpret_cast<uintptr_t>(o.p) & 15) == 0 && o.sb % 8 == 0 && o.st % 8 == 0 && o.sh % 8 == 0;
}

}  // namespace

// FULL, WIDE or SINGLE for x, B, C and up to two more operands of P features
int ssm_fit(const SsmArgs &a, const SsmOperand &p, const SsmOperand &q) {
    if (a.P % 8 || a.N % 8 || !wide(a.x) || !wide(a.Bm) || !wide(a.Cm) || !wide(p) || !wide(q)) return SINGLE;
    return a.P == 64 && (a.N == 32 || a.N == 64 || a.N == 128) ? FULL : WIDE;
}

bool ssm_mfma_supported(const SsmArgs &a) {
    return a.io == 1 && a.P <= 64 && a.N <= 128 && (reinterpret_cast<uintptr_t>(a.ws) & 15) == 0;
}

hipError_t launch_ssm_shares_mfma(const SsmArgs &a, const SsmOperand &dy, const float *prep, float *sf, float *sr,
                                  float *decay, hipStream_t stream) {
    MfmaArgs f{a, nullptr, 0, sf, decay, prep}, r{a, nullptr, 0, sr, nullptr, prep};
    r.a.x = dy;
    r.a.Bm = a.Cm;
    return run(ssm_fit(a, dy, dy), nullptr, &f, &r, stream);
}

hipError_t launch_ssm_mfma(const SsmArgs &a, hipStream_t stream) {
    const int64_t NP = static_cast<int64_t>(a.N) * a.P;
    const int fit = ssm_fit(a, a.y, a.y);
    float *prep = a.ws, *seg = a.ws + ssm_prep_floats(a.B, a.L, a.H);
    hipError_t e;
    if ((e = launch_ssm_prep(a, prep, stream)) != hipSuccess) return e;
    MfmaArgs w{a, a.state, 0, a.state_out, nullptr, prep};
    if (a.nseg > 1) {
        float *decay = seg + static_cast<int64_t>(a.B) * a.H * a.nseg * NP;
        const MfmaArgs p{a, nullptr, 0, seg, decay, prep};
        if ((e = run(fit, nullptr, &p, nullptr, stream)) != hipSuccess) return e;
        const SsmCarry c{a.state, decay, seg, a.state_out, 0};
        if ((e = launch_ssm_carry(a.B * a.H, static_cast<int>(NP), a.nseg, c, nullptr, stream)) != hipSuccess) return e;
        w.init = seg;
        w.init_stride = NP;
        w.fin = nullptr;
    }
    return run(fit, &w, nullptr, nullptr, stream);
}

}  // namespace ttt
