// The selective state space scan in fp32 vector arithmetic, for every head
// and state size up to 128 and both storage types. With u_t = D_t x_t and
// a_t = exp(D_t A), D_t = softplus(dt_t + dt_bias):
//     h_t = a_t h_{t-1} + B_t u_t^T,    y_t = C_t h_t + D x_t
// and the gradients, g_t the loss's gradient in h_t,
//     g_t = a_{t+1} g_{t+1} + C_t dy_t^T,
//     du_t = B_t g_t,   dB_t = g_t u_t,   dC_t = h_t dy_t.
// All are one walk: a state (key x value) gains k_t v_t^T and is read by a
// query over the keys,
//     y : k = B, v = u, q = C          dC : k = u, v = B, q = dy   (forwards)
//     du: k = C, v = dy, q = B         dB : k = dy, v = C, q = u   (backwards)
// so one kernel serves the four, with the state's two axes exchanged in dB
// and dC. One wave holds a whole state of up to 128 keys and 64 values: lane
// (g = lane / 16, c = lane % 16) has KPL = keys / 4 keys from g KPL on of
// VPL = values / 16 values from c VPL on. A token's keys and queries are read
// from LDS as 16-byte broadcasts that serve VPL products each; the sum over
// the keys is in the lane's registers and then over the four lane rows. No
// wave waits for another. The walk reads the state before the token's own
// k_t v_t^T is added where the gradient of the decay needs it ("strict"; the
// last term, (k_t . q_t) v_t, is added afterwards), else behind it.
//
// Vector bound: three fp32 operations for each token, key and value, one wave
// instruction each four cycles; tokens are staged T at a time, fetched to
// registers while the T before are worked on. Segments of the sequence run
// side by side (their states at the borders from a pass that does the update
// alone). B=3 L=517 H=6 P=48 N=24 fp32: outputs 10.4 us, the update alone 8.4 us,
// the carry between them 5.3 us; few waves, so latency of a token's chain.
//
// A single token (step) is bound by the state's bytes: 64 sequences of 32 heads
// of 64 x 64 read and write 67 MB in 12.7 us, 5.3 TB/s.
#include "ssm.hpp"
#include "vec.hpp"

namespace ttt {
namespace {

constexpr int T = 16;  // tokens staged at a time

enum Mode { STATES, STATES_REV, OUT_Y, OUT_DC, OUT_DU, OUT_DB };
constexpr bool reversed(int m) { return m == STATES_REV || m == OUT_DU || m == OUT_DB; }
constexpr bool exchanged(int m) { return m == OUT_DC || m == OUT_DB; }

struct WalkArgs {
    SsmArgs a;
    SsmOperand dy, dx;
    const float *init;  // [B,H,(nseg,)N,P] states that the walk starts from, or null (zeros)
    int64_t init_stride;  // floats between a head's segments (0: only one segment)
    float *fin;         // STATES: [B,H,nseg,N,P]; else the state after a single segment, or null
    float *decay;       // STATES: [B,H,nseg]
    float *per_head;    // OUT_DC, OUT_DB: [B,H,L,N]
    float *row, *col, *xdu, *dyx;  // per token sums, [value block][B,H,L]
};

template <typename TIO>
__device__ __forceinline__ float at(const SsmOperand &o, int b, int t, int h, int i) {
    return io_traits<TIO>::load(static_cast<const TIO *>(o.p), b * o.sb + t * o.st + h * o.sh + i);
}

template <int MODE, int KPL, int VPL, typename TIO>
__global__ __launch_bounds__(64) void walk(WalkArgs w) {
    const SsmArgs &a = w.a;
    constexpr bool REV = reversed(MODE), EX = exchanged(MODE), OUT = MODE >= OUT_Y;
    constexpr bool STRICT = MODE == OUT_DC || MODE == OUT_DU;
    constexpr int KP = 4 * KPL, VP = 16 * VPL, KN = T * KP / 64, VN = T * VP / 64;  // KN, VN: loads of T rows
    __shared__ alignas(16) float ks[T][KP], qs[OUT ? T : 1][KP], vs[T][VP];
    __shared__ float as[T], ds[T], dot[T];
    const int KD = EX ? a.P : a.N, VD = EX ? a.N : a.P;
    const int lane = threadIdx.x, g = lane / 16, c = lane % 16;
    const int vb = blockIdx.y, v0 = vb * VP;
    const int seg = blockIdx.x % a.nseg;
    const int bh = blockIdx.x / a.nseg, b = bh / a.H, h = bh % a.H, gr = h / (a.H / a.G);
    const int n = a.lens ? max(0, min(a.lens[b], a.L)) : a.L;
    const int64_t s0 = static_cast<int64_t>(seg) * a.seglen;
    const int t0 = static_cast<int>(s0 < a.L ? s0 : a.L);
    const int t1 = static_cast<int>(s0 + a.seglen < a.L ? s0 + a.seglen : a.L);
    const int te = max(t0, min(t1, n));  // tokens t0 .. te - 1 are walked
    const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f, Dh = a.D ? a.D[h] : 0.f;
    const int64_t NP = static_cast<int64_t>(a.N) * a.P;
    // keys, queries and values: rows of x or dy (of the head), of B or C (of the group)
    auto row = [&](const SsmOperand &o, int head) { return static_cast<const TIO *>(o.p) + b * o.sb + head * o.sh; };
    const bool kx = MODE == OUT_DC, ky = MODE == OUT_DB, kc = MODE == STATES_REV || MODE == OUT_DU;
    const SsmOperand &ok = kx ? a.x : ky ? w.dy : kc ? a.Cm : a.Bm;
    const SsmOperand &oq = MODE == OUT_Y ? a.Cm : MODE == OUT_DU ? a.Bm : MODE == OUT_DC ? w.dy : a.x;
    const SsmOperand &ov = MODE == OUT_DC ? a.Bm : MODE == OUT_DB ? a.Cm : REV ? w.dy : a.x;
    const TIO *kp = row(ok, EX ? h : gr), *qp = row(oq, EX ? h : gr), *vp = row(ov, EX ? gr : h);
    const TIO *dp = row(a.dt, h), *xp = row(a.x, h), *cp = row(a.Cm, gr);
    // element (key k, value v) of a state [N,P]
    auto place = [&](int k, int v) { return EX ? static_cast<int64_t>(v) * a.P + k : static_cast<int64_t>(k) * a.P + v; };
    float st[KPL][VPL];
    const float *init = w.init ? w.init + (w.init_stride ? w.init_stride * (static_cast<int64_t>(bh) * a.nseg + seg) : bh * NP) : nullptr;
#pragma unroll
    for (int i = 0; i < KPL; ++i)
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int k = g * KPL + i, v = v0 + c * VPL + j;
            st[i][j] = init && k < KD && v < VD ? init[place(k, v)] : 0.f;
        }
    // the value whose sum over the keys this lane receives
    const int vo = VPL == 4 ? 4 * c + g : VPL == 2 ? 2 * c + g / 2 : c;
    const bool own = v0 + vo < VD && (VPL == 4 || (VPL == 2 ? g % 2 == 0 : g == 0));
    float total = 0.f;  // sum of D_t A over the segment
    const int chunks = (te - t0 + T - 1) / T;
    float fk[KN], fq[OUT ? KN : 1], fv[VN], fd = 0.f;
    auto fetch = [&](int ci) {  // rows and columns past the end are read from the last and not used
        const int c0 = t0 + (REV ? chunks - 1 - ci : ci) * T, last = min(T, te - c0) - 1;
        fd = io_traits<TIO>::load(dp, static_cast<int64_t>(c0 + min(lane, last)) * a.dt.st);
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int64_t at = c0 + min((64 * i + lane) / KP, last);
            const int k = min((64 * i + lane) % KP, KD - 1);
            fk[i] = io_traits<TIO>::load(kp, at * ok.st + k);
            if (OUT) fq[i] = io_traits<TIO>::load(qp, at * oq.st + k);
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int64_t at = c0 + min((64 * i + lane) / VP, last);
            fv[i] = io_traits<TIO>::load(vp, at * ov.st + min(v0 + (64 * i + lane) % VP, VD - 1));
        }
    };
    if (chunks > 0) fetch(0);
    for (int ci = 0; ci < chunks; ++ci) {
        const int c0 = t0 + (REV ? chunks - 1 - ci : ci) * T, cn = min(T, te - c0);
        __syncthreads();  // the one wave has read what it staged before
        if (lane < T) {
            const float d = lane < cn ? softplus_f(fd + bias) : 0.f;
            ds[lane] = d;
            as[lane] = exp_f(at_least(d * A, -150.f));  // 0 below that
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int t = (64 * i + lane) / KP, k = (64 * i + lane) % KP;
            // u = D x wherever x enters as a key or a query
            const float d = EX ? ds[t] : 1.f;
            float kv = k < KD && t < cn ? fk[i] : 0.f, qv = OUT && k < KD ? fq[i] : 0.f;  // no key: adds nothing
            if (MODE == OUT_DC) kv *= d;
            if (MODE == OUT_DB) qv *= d;
            ks[t][k] = kv;
            if (OUT) qs[t][k] = qv;
        }
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int t = (64 * i + lane) / VP, v = (64 * i + lane) % VP;
            vs[t][v] = v0 + v < VD && t < cn ? fv[i] : 0.f;  // an infinity behind the end would be 0 x inf
        }
        if (STRICT) {  // k . q of each token: four lanes a token
            __syncthreads();
            float p = 0.f;
#pragma unroll 4
            for (int k = lane % 4; k < KP; k += 4) p = fmaf(ks[lane / 4][k], qs[lane / 4][k], p);
            p += __shfl_xor(p, 1, 64);
            p += __shfl_xor(p, 2, 64);
            if (lane % 4 == 0) dot[lane / 4] = p;
        }
        if (ci + 1 < chunks) fetch(ci + 1);
        __syncthreads();
        // all T, those past the end decay and add nothing: some tokens' LDS reads
        // are under way while one is worked on
#pragma unroll 2
        for (int i = 0; i < T; ++i) {
            const int t = REV ? T - 1 - i : i;
            const bool in = t < cn;
            const float dcy = as[t], dv = ds[t];
            total = fmaf(dv, A, total);
            float v[VPL], o[VPL] = {};
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                v[j] = vs[t][c * VPL + j];
                if (MODE == STATES || MODE == OUT_Y) v[j] *= dv;
            }
#pragma unroll
            for (int k = 0; k < KPL; ++k) {
                const float kk = ks[t][g * KPL + k], qq = OUT ? qs[t][g * KPL + k] : 0.f;
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    if (STRICT) {
                        if (!REV) st[k][j] *= dcy;
                        o[j] = fmaf(qq, st[k][j], o[j]);
                        st[k][j] = fmaf(kk, v[j], st[k][j]);
                    } else {
                        st[k][j] = REV ? fmaf(kk, v[j], st[k][j]) : fmaf(kk, v[j], st[k][j] * dcy);
                        if (OUT) o[j] = fmaf(qq, st[k][j], o[j]);
                    }
                    if (REV) st[k][j] *= dcy;
                }
            }
            if (OUT) {
                float out;
                if constexpr (VPL == 4)
                    out = tile::rows4_reduce4(o[0], o[1], o[2], o[3]);
                else if constexpr (VPL == 2)
                    out = tile::rows4_reduce2(o[0], o[1]);
                else
                    out = tile::rows4_sum(o[0]);
                const float raw = vs[t][vo];
                const int64_t tok = static_cast<int64_t>(bh) * a.L + c0 + t;
                const int64_t blk = static_cast<int64_t>(vb) * a.B * a.H * a.L + tok;
                if (MODE == OUT_Y && own && in)
                    io_traits<TIO>::store(static_cast<TIO *>(const_cast<void *>(a.y.p)),
                                          b * a.y.sb + (c0 + t) * a.y.st + h * a.y.sh + v0 + vo, fmaf(Dh, raw, out));
                if (MODE == OUT_DB && own && in) w.per_head[tok * a.N + v0 + vo] = out;
                if (MODE == OUT_DC) {  // raw = B
                    const float cv = own && in ? io_traits<TIO>::load(cp, (c0 + t) * a.Cm.st + v0 + vo) : 0.f;
                    if (own && in) w.per_head[tok * a.N + v0 + vo] = fmaf(dot[t], raw, out);
                    const float s = tile::rows4_sum(tile::row16_sum(cv * out));
                    if (lane == 0 && in) w.row[blk] = s;
                }
                if (MODE == OUT_DU) {  // raw = dy
                    const float du = fmaf(dot[t], raw, out);
                    const float x = own && in ? io_traits<TIO>::load(xp, (c0 + t) * a.x.st + v0 + vo) : 0.f;
                    if (own && in)
                        io_traits<TIO>::store(static_cast<TIO *>(const_cast<void *>(w.dx.p)),
                                              b * w.dx.sb + (c0 + t) * w.dx.st + h * w.dx.sh + v0 + vo,
                                              fmaf(dv, du, Dh * raw));
                    const float s = tile::rows4_sum(tile::row16_sum(x * out));
                    const float xu = tile::rows4_sum(tile::row16_sum(x * du));
                    const float yx = tile::rows4_sum(tile::row16_sum(x * raw));
                    if (lane == 0 && in) {
                        w.col[blk] = dv * s;
                        w.xdu[blk] = xu;
                        w.dyx[blk] = yx;
                    }
                }
            }
        }
    }
    // rows past the sequence's end are zeros
    if (OUT && lane < VP && v0 + lane < VD) {
        for (int t = te; t < t1; ++t) {
            const SsmOperand &o = MODE == OUT_Y ? a.y : w.dx;
            if (MODE == OUT_Y || MODE == OUT_DU)
                io_traits<TIO>::store(static_cast<TIO *>(const_cast<void *>(o.p)),
                                      b * o.sb + static_cast<int64_t>(t) * o.st + h * o.sh + v0 + lane, 0.f);
            else
                w.per_head[(static_cast<int64_t>(bh) * a.L + t) * a.N + v0 + lane] = 0.f;
        }
    }
    if (w.fin) {
        float *f = w.fin + (static_cast<int64_t>(bh) * (OUT ? 1 : a.nseg) + (OUT ? 0 : seg)) * NP;
#pragma unroll
        for (int i = 0; i < KPL; ++i)
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int k = g * KPL + i, v = v0 + c * VPL + j;
                if (k < KD && v < VD) f[place(k, v)] = st[i][j];
            }
    }
    if (!OUT && vb == 0 && lane == 0) w.decay[static_cast<int64_t>(bh) * a.nseg + seg] = exp_f(at_least(total, -150.f));
}

template <int MODE, int KPL, int VPL> hipError_t run_walk_kv(const WalkArgs &w, hipStream_t s) {
    const SsmArgs &a = w.a;
    const int VD = exchanged(MODE) ? a.N : a.P;
    const dim3 grid(static_cast<unsigned>(a.B) * a.H * a.nseg, (VD + 16 * VPL - 1) / (16 * VPL));
    if (a.io == 1)
        hipLaunchKernelGGL((walk<MODE, KPL, VPL, bf16_t>), grid, dim3(64), 0, s, w);
    else
        hipLaunchKernelGGL((walk<MODE, KPL, VPL, float>), grid, dim3(64), 0, s, w);
    return hipGetLastError();
}
template <int MODE, int KPL> hipError_t run_walk_k(const WalkArgs &w, hipStream_t s) {
    const int v = ssm_lane_values(w.a.B, w.a.L, w.a.H, exchanged(MODE) ? w.a.N : w.a.P);
    return v == 1 ? run_walk_kv<MODE, KPL, 1>(w, s) : v == 2 ? run_walk_kv<MODE, KPL, 2>(w, s) : run_walk_kv<MODE, KPL, 4>(w, s);
}
template <int MODE> hipError_t run_walk(const WalkArgs &w, hipStream_t s) {
    const int KD = exchanged(MODE) ? w.a.P : w.a.N;
    return KD <= 16   ? run_walk_k<MODE, 4>(w, s)
           : KD <= 32 ? run_walk_k<MODE, 8>(w, s)
           : KD <= 64 ? run_walk_k<MODE, 16>(w, s)
                      : run_walk_k<MODE, 32>(w, s);
}

constexpr int CT = 256;

// blockIdx.z: one walk over a head's segments, or a second one
__global__ __launch_bounds__(CT) void carry(int NP, int nseg, SsmCarry c0, SsmCarry c1) {
    const SsmCarry &c = blockIdx.z ? c1 : c0;
    const int i = blockIdx.x * CT + threadIdx.x;
    const int64_t bh = blockIdx.y;
    if (i >= NP) return;
    float *p = c.seg + bh * nseg * NP + i;
    const float *d = c.decay + bh * nseg;
    float s = c.first ? c.first[bh * NP + i] : 0.f;
    constexpr int U = 16;  // segments in flight
    for (int k0 = 0; k0 < nseg; k0 += U) {
        float v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = min(k0 + u, nseg - 1);
            v[u] = p[static_cast<int64_t>(c.reverse ? nseg - 1 - k : k) * NP];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k0 + u >= nseg) break;
            const int k = c.reverse ? nseg - 1 - (k0 + u) : k0 + u;
            p[static_cast<int64_t>(k) * NP] = s;
            s = fmaf(d[k], s, v[u]);
        }
    }
    if (c.out) c.out[bh * NP + i] = s;
}

// one token: the state is read, updated and written in place
constexpr int ST = 256;
template <int V, typename TIO>
__global__ __launch_bounds__(ST) void step(SsmArgs a, int lpr) {
    __shared__ float red[ST * V];
    const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H, gr = h / (a.H / a.G);
    const int row = threadIdx.x / lpr, p0 = (threadIdx.x % lpr) * V, rows = ST / lpr;
    const bool in = p0 < a.P;
    const float d = softplus_f(at<TIO>(a.dt, b, 0, h, 0) + (a.dt_bias ? a.dt_bias[h] : 0.f));
    const float dcy = expf(d * a.A[h]);
    float x[V], y[V] = {};
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = in ? at<TIO>(a.x, b, 0, h, p0 + v) : 0.f;
    float *s = a.state_out + static_cast<int64_t>(bh) * a.N * a.P + p0;
    constexpr int U = 4;
    for (int n0 = row; n0 < a.N; n0 += U * rows) {
        float hv[U][V], Bv[U], Cv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int n = n0 + u * rows;
            if (in && n < a.N) {
                vec_load<float, V>(s + static_cast<int64_t>(n) * a.P, hv[u]);
                Bv[u] = at<TIO>(a.Bm, b, 0, gr, n);
                Cv[u] = at<TIO>(a.Cm, b, 0, gr, n);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int n = n0 + u * rows;
            if (in && n < a.N) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    hv[u][v] = fmaf(dcy, hv[u][v], Bv[u] * (d * x[v]));
                    y[v] = fmaf(Cv[u], hv[u][v], y[v]);
                }
                VecIO<float, V>::store(s + static_cast<int64_t>(n) * a.P, hv[u]);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) red[(row * lpr + threadIdx.x % lpr) * V + v] = y[v];
    __syncthreads();
    const int w = lpr * V;
    for (int p = threadIdx.x; p < a.P; p += ST) {
        float v = 0.f;
        for (int r = 0; r < rows; ++r) v += red[r * w + p];
        if (a.D) v = fmaf(a.D[h], at<TIO>(a.x, b, 0, h, p), v);
        io_traits<TIO>::store(static_cast<TIO *>(const_cast<void *>(a.y.p)), static_cast<int64_t>(bh) * a.P + p, v);
    }
}

template <typename TIO> hipError_t step_t(const SsmArgs &a, hipStream_t s) {
    const bool vec = a.P % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state_out) & 15) == 0;
    int lpr = 1;
    while (lpr * (vec ? 4 : 1) < a.P) lpr *= 2;
    if (vec)
        hipLaunchKernelGGL((step<4, TIO>), dim3(static_cast<unsigned>(a.B) * a.H), dim3(ST), 0, s, a, lpr);
    else
        hipLaunchKernelGGL((step<1, TIO>), dim3(static_cast<unsigned>(a.B) * a.H), dim3(ST), 0, s, a, lpr);
    return hipGetLastError();
}

}  // namespace

// Values of a lane: as many as a row of LDS reads can serve, fewer where that
// leaves SIMDs without a wave, as a lone wave is bound by its own instructions
// (B = 3, H = 6, N = 24, P = 48, 517 tokens: outputs 15.9 us with 4 values a
// lane, 10.4 us with 1). Goes by the sizes alone, as the workspace does.
int ssm_lane_values(int B, int L, int H, int VD) {
    const int64_t units = static_cast<int64_t>(B) * H * ((static_cast<int64_t>(L) + 63) / 64);
    if (VD <= 16 || units * ((VD + 31) / 32) < 512) return 1;
    return VD <= 32 || units * ((VD + 63) / 64) < 512 ? 2 : 4;
}

hipError_t launch_ssm_step(const SsmArgs &a, hipStream_t stream) {
    return a.io == 1 ? step_t<bf16_t>(a, stream) : step_t<float>(a, stream);
}

hipError_t launch_ssm_carry(int BH, int NP, int nseg, const SsmCarry &c, const SsmCarry *other, hipStream_t stream) {
    for (int h0 = 0; h0 < BH; h0 += 65535) {  // a grid has at most 65535 rows
        const int nh = BH - h0 < 65535 ? BH - h0 : 65535;
        auto from = [&](SsmCarry x) {
            const int64_t o = static_cast<int64_t>(h0) * NP;
            x.first = x.first ? x.first + o : nullptr;
            x.out = x.out ? x.out + o : nullptr;
            x.decay += static_cast<int64_t>(h0) * nseg;
            x.seg += o * nseg;
            return x;
        };
        hipLaunchKernelGGL(carry, dim3((NP + CT - 1) / CT, nh, other ? 2 : 1), dim3(CT), 0, stream, NP, nseg,
                           from(c), from(other ? *other : c));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_ssm_states_valu(const SsmArgs &a, const SsmOperand *dy, float *seg, float *decay,
                                  hipStream_t stream) {
    WalkArgs w{};
    w.a = a;
    w.fin = seg;
    w.decay = decay;
    if (!dy) return run_walk<STATES>(w, stream);
    w.dy = *dy;
    return run_walk<STATES_REV>(w, stream);
}

hipError_t launch_ssm_forward(const SsmArgs &a, hipStream_t stream) {
    hipError_t e;
    const int64_t NP = static_cast<int64_t>(a.N) * a.P;
    if (ssm_mfma_supported(a)) return launch_ssm_mfma(a, stream);
    WalkArgs w{};
    w.a = a;
    if (a.nseg > 1) {
        float *seg = a.ws, *decay = a.ws + static_cast<int64_t>(a.B) * a.H * a.nseg * NP;
        if ((e = launch_ssm_states_valu(a, nullptr, seg, decay, stream)) != hipSuccess) return e;
        const SsmCarry c{a.state, decay, seg, a.state_out, 0};
        if ((e = launch_ssm_carry(a.B * a.H, static_cast<int>(NP), a.nseg, c, nullptr, stream)) != hipSuccess) return e;
        w.init = seg;
        w.init_stride = NP;
    } else {
        w.init = a.state;
        w.fin = a.state_out;
    }
    return run_walk<OUT_Y>(w, stream);
}

hipError_t launch_ssm_backward(const SsmBwdArgs &g, hipStream_t stream) {
    const SsmArgs &a = g.f;
    const int64_t NP = static_cast<int64_t>(a.N) * a.P;
    const SsmBwdWs s = ssm_backward_ws(a);
    hipError_t e;
    if (!a.B) return launch_ssm_bwd_finish(g, false, stream);  // the sums over no tokens
    if (ssm_bwd_mfma_supported(g)) return launch_ssm_bwd_mfma(g, stream);
    if ((e = launch_ssm_states_valu(a, nullptr, s.sf, s.decay, stream)) != hipSuccess) return e;
    if ((e = launch_ssm_states_valu(a, &g.dy, s.sr, s.decay, stream)) != hipSuccess) return e;
    const SsmCarry cf{a.state, s.decay, s.sf, s.last, 0}, cr{g.dstate_out, s.decay, s.sr, g.dstate, 1};
    if ((e = launch_ssm_carry(a.B * a.H, static_cast<int>(NP), a.nseg, cf, &cr, stream)) != hipSuccess) return e;
    WalkArgs w{};
    w.a = a;
    w.dy = g.dy;
    w.dx = g.dx;
    w.init_stride = NP;
    w.row = s.row;
    w.col = s.col;
    w.xdu = s.xdu;
    w.dyx = s.dyx;
    w.init = s.sf;
    w.per_head = s.dCh;
    if ((e = run_walk<OUT_DC>(w, stream)) != hipSuccess) return e;
    w.init = s.sr;
    if ((e = run_walk<OUT_DU>(w, stream)) != hipSuccess) return e;
    w.per_head = s.dBh;
    if ((e = run_walk<OUT_DB>(w, stream)) != hipSuccess) return e;
    return launch_ssm_bwd_finish(g, false, stream);
}

}  // namespace ttt
