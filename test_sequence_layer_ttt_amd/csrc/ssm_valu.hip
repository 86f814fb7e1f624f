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
// and dC. Lanes hold 64 values, each wave 16 keys of them in registers; a
// token's reads of k and q are LDS broadcasts. The walk reads the state
// before the token's own k_t v_t^T is added ("strict"); that last term is
// (k_t . q_t) v_t and is added afterwards, which also leaves the strict part
// to the gradient of the decay.
//
// Vector bound: three fp32 operations for each token, key and value, one wave
// instruction each four cycles. Segments of the sequence run side by side
// (their states at the borders from a pass that does the update alone).
#include "ssm.hpp"
#include "vec.hpp"

namespace ttt {
namespace {

constexpr int T = 16;   // tokens staged at a time
constexpr int KW = 16;  // keys of a wave

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

template <int MODE, typename TIO>
__global__ __launch_bounds__(512) void walk(WalkArgs w) {
    const SsmArgs &a = w.a;
    extern __shared__ float lds[];
    constexpr bool REV = reversed(MODE), EX = exchanged(MODE);
    constexpr bool OUT = MODE >= OUT_Y;
    const int KD = EX ? a.P : a.N, VD = EX ? a.N : a.P;
    const int nw = blockDim.x / 64, kp = nw * KW;
    float *ks = lds, *qs = ks + T * kp, *vs = qs + (OUT ? T * kp : 0), *as = vs + T * 64, *ds = as + T;
    float *yp = ds + T, *kq = yp + (OUT ? nw * T * 64 : 0);  // [nw][T][64], [nw][T]
    const int lane = threadIdx.x % 64, wv = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int vb = blockIdx.y, vi = vb * 64 + lane;
    const int seg = blockIdx.x % a.nseg;
    const int bh = blockIdx.x / a.nseg, b = bh / a.H, h = bh % a.H, gr = h / (a.H / a.G);
    const int n = a.lens ? max(0, min(a.lens[b], a.L)) : a.L;
    const int64_t s0 = static_cast<int64_t>(seg) * a.seglen;
    const int t0 = static_cast<int>(s0 < a.L ? s0 : a.L);
    const int t1 = static_cast<int>(s0 + a.seglen < a.L ? s0 + a.seglen : a.L);
    const int te = max(t0, min(t1, n));  // tokens t0 .. te - 1 are walked
    const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f;
    const int64_t NP = static_cast<int64_t>(a.N) * a.P;
    // element (key k, value v) of a state [N,P]
    auto place = [&](int k) { return EX ? static_cast<int64_t>(vi) * a.P + k : static_cast<int64_t>(k) * a.P + vi; };
    float st[KW];
#pragma unroll
    for (int i = 0; i < KW; ++i) {
        const int k = wv * KW + i;
        st[i] = 0.f;
        if (w.init && k < KD && vi < VD)
            st[i] = w.init[w.init_stride * (static_cast<int64_t>(bh) * a.nseg + seg) + (w.init_stride ? 0 : bh * NP) + place(k)];
    }
    float total = 0.f;  // sum of D_t A over the segment
    const int chunks = (te - t0 + T - 1) / T;
    for (int ci = 0; ci < chunks; ++ci) {
        const int c0 = t0 + (REV ? chunks - 1 - ci : ci) * T, cn = min(T, te - c0);
        __syncthreads();
        if (threadIdx.x < T) {
            float d = 0.f;
            if (static_cast<int>(threadIdx.x) < cn) d = softplus_f(at<TIO>(a.dt, b, c0 + threadIdx.x, h, 0) + bias);
            ds[threadIdx.x] = d;
            as[threadIdx.x] = expf(d * A);
        }
        for (int i = threadIdx.x; i < T * kp; i += blockDim.x) {
            const int t = i / kp, k = i % kp;
            float kv = 0.f, qv = 0.f;
            if (t < cn && k < KD) {
                if (MODE == STATES || MODE == OUT_Y) kv = at<TIO>(a.Bm, b, c0 + t, gr, k);
                if (MODE == STATES_REV || MODE == OUT_DU) kv = at<TIO>(a.Cm, b, c0 + t, gr, k);
                if (MODE == OUT_DC) kv = at<TIO>(a.x, b, c0 + t, h, k);
                if (MODE == OUT_DB) kv = at<TIO>(w.dy, b, c0 + t, h, k);
                if (MODE == OUT_Y) qv = at<TIO>(a.Cm, b, c0 + t, gr, k);
                if (MODE == OUT_DU) qv = at<TIO>(a.Bm, b, c0 + t, gr, k);
                if (MODE == OUT_DC) qv = at<TIO>(w.dy, b, c0 + t, h, k);
                if (MODE == OUT_DB) qv = at<TIO>(a.x, b, c0 + t, h, k);
            }
            ks[i] = kv;
            if (OUT) qs[i] = qv;
        }
        for (int i = threadIdx.x; i < T * 64; i += blockDim.x) {
            const int t = i / 64, v = vb * 64 + i % 64;
            float x = 0.f;
            if (t < cn && v < VD) {
                if (MODE == STATES || MODE == OUT_Y) x = at<TIO>(a.x, b, c0 + t, h, v);
                if (MODE == STATES_REV || MODE == OUT_DU) x = at<TIO>(w.dy, b, c0 + t, h, v);
                if (MODE == OUT_DC) x = at<TIO>(a.Bm, b, c0 + t, gr, v);
                if (MODE == OUT_DB) x = at<TIO>(a.Cm, b, c0 + t, gr, v);
            }
            vs[i] = x;
        }
        __syncthreads();
        for (int i = 0; i < cn; ++i) {
            const int t = REV ? cn - 1 - i : i;
            const float dcy = as[t], dv = ds[t];
            total = fmaf(dv, A, total);
            // u = D x wherever x enters: as value, key or query
            float v = vs[t * 64 + lane];
            if (MODE == STATES || MODE == OUT_Y) v *= dv;
            float o = 0.f, dot = 0.f;
#pragma unroll
            for (int j = 0; j < KW; ++j) {
                float k = ks[t * kp + wv * KW + j];
                if (MODE == OUT_DC) k *= dv;
                if (!REV) st[j] *= dcy;
                if (OUT) {
                    float q = qs[t * kp + wv * KW + j];
                    if (MODE == OUT_DB) q *= dv;
                    o = fmaf(q, st[j], o);
                    dot = fmaf(q, k, dot);
                }
                st[j] = fmaf(k, v, st[j]);
                if (REV) st[j] *= dcy;
            }
            if (OUT) {
                yp[(wv * T + t) * 64 + lane] = o;
                if (lane == 0) kq[wv * T + t] = dot;
            }
        }
        if (OUT) {
            __syncthreads();
            for (int t = wv; t < cn; t += nw) {
                float strict = 0.f, dot = 0.f;
                for (int i = 0; i < nw; ++i) {
                    strict += yp[(i * T + t) * 64 + lane];
                    dot += kq[i * T + t];
                }
                const float raw = vs[t * 64 + lane], dv = ds[t];
                const int64_t tok = static_cast<int64_t>(bh) * a.L + c0 + t;
                const int64_t blk = static_cast<int64_t>(vb) * a.B * a.H * a.L + tok;
                const bool in = vi < VD;
                if (MODE == OUT_Y) {
                    const float y = fmaf(dot, dv * raw, strict) + (a.D ? a.D[h] * raw : 0.f);
                    if (in)
                        io_traits<TIO>::store(static_cast<TIO *>(const_cast<void *>(a.y.p)),
                                              b * a.y.sb + (c0 + t) * a.y.st + h * a.y.sh + vi, y);
                }
                if (MODE == OUT_DC) {  // raw = B
                    if (in) w.per_head[tok * a.N + vi] = fmaf(dot, raw, strict);
                    const float s = tile::rows4_sum(tile::row16_sum(in ? at<TIO>(a.Cm, b, c0 + t, gr, vi) * strict : 0.f));
                    if (lane == 0) w.row[blk] = s;
                }
                if (MODE == OUT_DB) {  // raw = C
                    if (in) w.per_head[tok * a.N + vi] = fmaf(dot, raw, strict);
                }
                if (MODE == OUT_DU) {  // raw = dy
                    const float du = fmaf(dot, raw, strict);
                    const float x = in ? at<TIO>(a.x, b, c0 + t, h, vi) : 0.f;
                    if (in)
                        io_traits<TIO>::store(static_cast<TIO *>(const_cast<void *>(w.dx.p)),
                                              b * w.dx.sb + (c0 + t) * w.dx.st + h * w.dx.sh + vi,
                                              fmaf(dv, du, a.D ? a.D[h] * raw : 0.f));
                    const float c = tile::rows4_sum(tile::row16_sum(x * strict));
                    const float xu = tile::rows4_sum(tile::row16_sum(x * du));
                    const float yx = tile::rows4_sum(tile::row16_sum(x * raw));
                    if (lane == 0) {
                        w.col[blk] = dv * c;
                        w.xdu[blk] = xu;
                        w.dyx[blk] = yx;
                    }
                }
            }
        }
    }
    // rows past the sequence's end are zeros
    if (OUT) {
        for (int t = te + wv; t < t1; t += nw) {
            const int64_t tok = static_cast<int64_t>(bh) * a.L + t;
            const SsmOperand &o = MODE == OUT_Y ? a.y : w.dx;
            if (vi < VD) {
                if (MODE == OUT_Y || MODE == OUT_DU)
                    io_traits<TIO>::store(static_cast<TIO *>(const_cast<void *>(o.p)), b * o.sb + t * o.st + h * o.sh + vi, 0.f);
                else
                    w.per_head[tok * a.N + vi] = 0.f;
            }
        }
    }
    if (w.fin) {
        float *f = w.fin + (static_cast<int64_t>(bh) * (OUT ? 1 : a.nseg) + (OUT ? 0 : seg)) * NP;
#pragma unroll
        for (int i = 0; i < KW; ++i) {
            const int k = wv * KW + i;
            if (k < KD && vi < VD) f[place(k)] = st[i];
        }
    }
    if (!OUT && vb == 0 && threadIdx.x == 0) w.decay[static_cast<int64_t>(bh) * a.nseg + seg] = expf(total);
}

template <int MODE, typename TIO> hipError_t run_walk(const WalkArgs &w, hipStream_t s) {
    const SsmArgs &a = w.a;
    const int KD = exchanged(MODE) ? a.P : a.N, VD = exchanged(MODE) ? a.N : a.P;
    const int nw = (KD + KW - 1) / KW, kp = nw * KW;
    constexpr bool OUT = MODE >= OUT_Y;
    const size_t floats = T * kp * (OUT ? 2 : 1) + T * 64 + 2 * T + (OUT ? nw * T * 64 + nw * T : 0);
    hipLaunchKernelGGL((walk<MODE, TIO>), dim3(static_cast<unsigned>(a.B) * a.H * a.nseg, (VD + 63) / 64),
                       dim3(64 * nw), floats * sizeof(float), s, w);
    return hipGetLastError();
}
template <int MODE> hipError_t run_walk(const WalkArgs &w, hipStream_t s) {
    return w.a.io == 1 ? run_walk<MODE, bf16_t>(w, s) : run_walk<MODE, float>(w, s);
}

constexpr int CT = 256;

__global__ __launch_bounds__(CT) void carry(int NP, int nseg, int reverse, const float *first,
                                            const float *decay, float *seg, float *out) {
    const int i = blockIdx.x * CT + threadIdx.x;
    const int64_t bh = blockIdx.y;
    if (i >= NP) return;
    float *p = seg + bh * nseg * NP + i;
    const float *d = decay + bh * nseg;
    float s = first ? first[bh * NP + i] : 0.f;
    constexpr int U = 16;  // segments in flight
    for (int k0 = 0; k0 < nseg; k0 += U) {
        float v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = min(k0 + u, nseg - 1);
            v[u] = p[static_cast<int64_t>(reverse ? nseg - 1 - k : k) * NP];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k0 + u >= nseg) break;
            const int k = reverse ? nseg - 1 - (k0 + u) : k0 + u;
            p[static_cast<int64_t>(k) * NP] = s;
            s = fmaf(d[k], s, v[u]);
        }
    }
    if (out) out[bh * NP + i] = s;
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

hipError_t launch_ssm_step(const SsmArgs &a, hipStream_t stream) {
    return a.io == 1 ? step_t<bf16_t>(a, stream) : step_t<float>(a, stream);
}

hipError_t launch_ssm_carry(int BH, int NP, int nseg, bool reverse, const float *first, const float *decay,
                            float *seg, float *out, hipStream_t stream) {
    for (int h0 = 0; h0 < BH; h0 += 65535) {  // a grid has at most 65535 rows
        const int nh = BH - h0 < 65535 ? BH - h0 : 65535;
        const int64_t o = static_cast<int64_t>(h0) * NP;
        hipLaunchKernelGGL(carry, dim3((NP + CT - 1) / CT, nh), dim3(CT), 0, stream, NP, nseg, reverse ? 1 : 0,
                           first ? first + o : nullptr, decay + static_cast<int64_t>(h0) * nseg, seg + o * nseg,
                           out ? out + o : nullptr);
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
        if ((e = launch_ssm_carry(a.B * a.H, static_cast<int>(NP), a.nseg, false, a.state, decay, seg,
                                  a.state_out, stream)) != hipSuccess)
            return e;
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
    if ((e = launch_ssm_carry(a.B * a.H, static_cast<int>(NP), a.nseg, false, a.state, s.decay, s.sf, s.last,
                              stream)) != hipSuccess)
        return e;
    if ((e = launch_ssm_states_valu(a, &g.dy, s.sr, s.decay, stream)) != hipSuccess) return e;
    if ((e = launch_ssm_carry(a.B * a.H, static_cast<int>(NP), a.nseg, true, g.dstate_out, s.decay, s.sr,
                              g.dstate, stream)) != hipSuccess)
        return e;
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
