// extern "C" entry points of the operators around the layer (declared and
// documented in ttt.h): validation on the host, then the launch. Nothing here
// allocates or synchronises.
#include <algorithm>
#include <utility>

#include "abi_common.hpp"
#include "block.hpp"
#include "ssm.hpp"

using namespace ttt::abi;

namespace {

// A strided operand of up to two rows' dimensions (batch, token), a head
// dimension and a contiguous innermost one. Strides are in elements.
struct View {
    const void *p;
    const char *name;
    int64_t nb, nt, nh, inner;  // sizes
    int64_t sb, st, sh;         // strides
    unsigned es;                // bytes of an element
};

// the strides a NULL array stands for: row-major and contiguous
View view(const void *p, const char *name, int64_t nb, int64_t nt, int64_t nh, int64_t inner,
          const int64_t *strides, int rank, unsigned es) {
    View v{p, name, nb, nt, nh, inner, nt * nh * inner, nh * inner, inner, es};
    if (strides) {
        v.sb = strides[0];
        if (rank > 1) v.st = strides[1];
        if (rank > 2) v.sh = strides[2];
    }
    return v;
}

bool empty(const View &v) { return !v.nb || !v.nt || !v.nh || !v.inner; }

// bytes from the first to behind the last element; false on overflow
bool extent(const View &v, size_t *out) {
    if (empty(v)) {
        *out = 0;
        return true;
    }
    int64_t n = v.inner;
    const int64_t dims[3][2] = {{v.nb, v.sb}, {v.nt, v.st}, {v.nh, v.sh}};
    for (const auto &d : dims) {
        int64_t m;
        if (__builtin_mul_overflow(d[0] - 1, d[1], &m) || __builtin_add_overflow(n, m, &n)) return false;
    }
    int64_t bytes;
    if (__builtin_mul_overflow(n, static_cast<int64_t>(v.es), &bytes)) return false;
    *out = static_cast<size_t>(bytes);
    return true;
}

int check_view(const View &v, bool out, size_t *bytes) {
    if (v.sb < 0 || v.st < 0 || v.sh < 0)
        return fail(TTT_E_SHAPE, "%s has a negative stride", v.name);
    if (!extent(v, bytes)) return fail(TTT_E_SHAPE, "sizes of %s overflow", v.name);
    if (!v.p) {
        if (*bytes) return fail(TTT_E_NULL, "%s is NULL (%zu bytes expected)", v.name, *bytes);
        return TTT_OK;
    }
    if (reinterpret_cast<uintptr_t>(v.p) & (v.es - 1))
        return fail(TTT_E_ALIGN, "%s (%p) is not %u-byte aligned", v.name, v.p, v.es);
    if (out && *bytes) {  // every element at an address of its own
        std::pair<int64_t, int64_t> d[3] = {{v.sb, v.nb}, {v.st, v.nt}, {v.sh, v.nh}};
        std::sort(d, d + 3);
        int64_t below = v.inner;
        for (const auto &x : d) {
            if (x.second == 1) continue;
            if (x.first < below) return fail(TTT_E_SHAPE, "elements of the output %s share addresses", v.name);
            below += (x.second - 1) * x.first;
        }
    }
    return TTT_OK;
}

// Whether two views whose extents overlap still have no byte in common: both
// are columns of the same rows (equal batch and token strides, rows that do
// not reach past a token's stride).
bool apart(const View &a, const View &b) {
    if (a.es != b.es || a.nb != b.nb || a.nt != b.nt) return false;
    const int64_t wa = (a.nh - 1) * a.sh + a.inner, wb = (b.nh - 1) * b.sh + b.inner;
    int64_t row;
    if (a.nt > 1) {
        if (a.st != b.st || (a.nb > 1 && (a.sb != b.sb || a.sb % a.st))) return false;
        row = a.st;
    } else {
        if (a.nb > 1 && a.sb != b.sb) return false;
        row = a.nb > 1 ? a.sb : INT64_MAX;
    }
    const char *pa = static_cast<const char *>(a.p), *pb = static_cast<const char *>(b.p);
    const bool first = pa <= pb;
    const int64_t d = (first ? pb - pa : pa - pb) / a.es;
    return d >= (first ? wa : wb) && d + (first ? wb : wa) <= row;
}

struct Views {
    View v[20];
    size_t bytes[20];
    bool out[20];
    int n = 0;
    int add(const View &x, bool output) {
        const int st = check_view(x, output, &bytes[n]);
        v[n] = x;
        out[n++] = output;
        return st;
    }
    int add_in(const View &x) { return add(x, false); }
    int add_out(const View &x) { return add(x, true); }
    // outputs against everything before and behind them; `same`: an output
    // that may be exactly the input it replaces
    int alias(const void *same_out = nullptr, const void *same_in = nullptr) const {
        for (int o = 0; o < n; ++o) {
            if (!out[o] || !v[o].p || !bytes[o]) continue;
            for (int i = 0; i < n; ++i) {
                if (i == o || (out[i] && i < o) || !v[i].p || !bytes[i]) continue;
                const uintptr_t a = reinterpret_cast<uintptr_t>(v[o].p), b = reinterpret_cast<uintptr_t>(v[i].p);
                if (a >= b + bytes[i] || b >= a + bytes[o]) continue;
                if (same_out && v[o].p == same_out && v[i].p == same_in && same_out == same_in &&
                    bytes[o] == bytes[i] && !out[i])
                    continue;
                if (apart(v[o], v[i])) continue;
                return fail(TTT_E_ALIAS, "%s overlaps %s", v[o].name, v[i].name);
            }
        }
        return TTT_OK;
    }
};

View flat(const void *p, const char *name, int64_t n, unsigned es) {
    return view(p, name, 1, 1, 1, n, nullptr, 0, es);
}

int check_sizes(int B, int L, int io) {
    if (B < 0 || L < 0) return fail(TTT_E_SHAPE, "negative size (B=%d L=%d)", B, L);
    if (io != TTT_F32 && io != TTT_BF16) return fail(TTT_E_DTYPE, "io dtype %d is not TTT_F32/TTT_BF16", io);
    if (L > TTT_MAX_L) return fail(TTT_E_SHAPE, "L = %d exceeds TTT_MAX_L = %d", L, TTT_MAX_L);
    return TTT_OK;
}

constexpr int MAX_GRID_YZ = 65535;

int conv_common(int B, int L, int C, int K, int io, int act) {
    int st;
    if ((st = check_sizes(B, L, io))) return st;
    if (C < 0 || C > TTT_CONV_MAX_C) return fail(TTT_E_SHAPE, "C = %d not in [0, %d]", C, TTT_CONV_MAX_C);
    if (K < 2 || K > 4) return fail(TTT_E_SHAPE, "K = %d not in [2, 4]", K);
    if (act != TTT_ACT_NONE && act != TTT_ACT_SILU)
        return fail(TTT_E_SHAPE, "activation %d is not TTT_ACT_NONE / TTT_ACT_SILU", act);
    return TTT_OK;
}

unsigned esize(int io) { return io == TTT_BF16 ? 2 : 4; }

}  // namespace

extern "C" {

int ttt_conv_forward(int B, int L, int C, int K, int io, int act, const void *x, const int64_t *x_strides,
                     const float *weight, const float *bias, const void *state, const int *lens, void *y,
                     const int64_t *y_strides, void *state_out, hipStream_t stream) {
    int st;
    if ((st = conv_common(B, L, C, K, io, act))) return st;
    if (B > MAX_GRID_YZ) return fail(TTT_E_SHAPE, "B = %d exceeds %d", B, MAX_GRID_YZ);
    const unsigned es = esize(io);
    const View vx = view(x, "x", B, L, 1, C, x_strides, 2, es), vy = view(y, "y", B, L, 1, C, y_strides, 2, es);
    const int64_t sn = static_cast<int64_t>(B) * (K - 1) * C;
    Views v;
    if ((st = v.add_in(vx)) || (st = v.add_in(flat(weight, "weight", static_cast<int64_t>(C) * K, 4))) ||
        (st = v.add_in(flat(bias, "bias", bias ? C : 0, 4))) ||
        (st = v.add_in(flat(state, "state", state ? sn : 0, es))) ||
        (st = v.add_in(flat(lens, "lens", lens ? B : 0, 4))) || (st = v.add_out(vy)) ||
        (st = v.add_out(flat(state_out, "state_out", state_out ? sn : 0, es))) ||
        (st = v.alias(state_out, state)))
        return st;
    if (!B || !C || (!L && !state_out)) return ok();
    ttt::ConvArgs a{B, L, C, K, io, act == TTT_ACT_SILU, x, vx.sb, vx.st, weight, bias, state, lens,
                    y, vy.sb, vy.st, state_out};
    return launched(ttt::launch_conv_forward(a, stream));
}

int ttt_conv_step(int B, int C, int K, int io, int act, const void *x, const int64_t *x_strides,
                  const float *weight, const float *bias, void *state, void *y, hipStream_t stream) {
    int st;
    if ((st = conv_common(B, 1, C, K, io, act))) return st;
    const unsigned es = esize(io);
    const View vx = view(x, "x", B, 1, 1, C, x_strides, 1, es), vy = view(y, "y", B, 1, 1, C, nullptr, 0, es);
    if (static_cast<int64_t>(B) * C > INT_MAX) return fail(TTT_E_SHAPE, "B*C too large");
    Views v;
    if ((st = v.add_in(vx)) || (st = v.add_in(flat(weight, "weight", static_cast<int64_t>(C) * K, 4))) ||
        (st = v.add_in(flat(bias, "bias", bias ? C : 0, 4))) ||
        (st = v.add_out(flat(state, "state", static_cast<int64_t>(B) * (K - 1) * C, es))) ||
        (st = v.add_out(vy)) || (st = v.alias()))
        return st;
    if (!B || !C) return ok();
    ttt::ConvArgs a{B, 1, C, K, io, act == TTT_ACT_SILU, x, vx.sb, vx.st, weight, bias, nullptr, nullptr,
                    y, vy.sb, vy.st, state};
    return launched(ttt::launch_conv_step(a, stream));
}

int ttt_conv_backward_workspace(int B, int L, int C, int K, size_t *bytes) {
    int st;
    if ((st = conv_common(B, L, C, K, TTT_F32, TTT_ACT_NONE))) return st;
    if (!bytes) return fail(TTT_E_NULL, "bytes is NULL");
    const int64_t rows = ttt::conv_backward_blocks(B, L, C);
    if (B > MAX_GRID_YZ || rows > INT_MAX) return fail(TTT_E_SHAPE, "B = %d or B*L is too large", B);
    *bytes = static_cast<size_t>(rows) * static_cast<size_t>(C) * static_cast<size_t>(K + 1) * sizeof(float);
    return ok();
}

int ttt_conv_backward(int B, int L, int C, int K, int io, int act, const void *x, const int64_t *x_strides,
                      const float *weight, const float *bias, const void *state, const int *lens,
                      const void *dy, const int64_t *dy_strides, const void *dstate_out, void *dx,
                      const int64_t *dx_strides, float *dweight, float *dbias, void *dstate, void *workspace,
                      size_t workspace_bytes, hipStream_t stream) {
    int st;
    size_t need;
    if ((st = conv_common(B, L, C, K, io, act)) || (st = ttt_conv_backward_workspace(B, L, C, K, &need))) return st;
    if ((dbias != nullptr) != (bias != nullptr) && C)
        return fail(TTT_E_NULL, "dbias is given exactly when bias is");
    const int64_t sn = static_cast<int64_t>(B) * (K - 1) * C;
    if ((dstate != nullptr) != (state != nullptr) && sn)
        return fail(TTT_E_NULL, "dstate is given exactly when state is");
    const unsigned es = esize(io);
    const View vx = view(x, "x", B, L, 1, C, x_strides, 2, es), vd = view(dy, "dy", B, L, 1, C, dy_strides, 2, es),
               vo = view(dx, "dx", B, L, 1, C, dx_strides, 2, es);
    const int64_t wn = static_cast<int64_t>(C) * K;
    Views v;
    if ((st = v.add_in(vx)) || (st = v.add_in(flat(weight, "weight", wn, 4))) ||
        (st = v.add_in(flat(bias, "bias", bias ? C : 0, 4))) ||
        (st = v.add_in(flat(state, "state", state ? sn : 0, es))) ||
        (st = v.add_in(flat(lens, "lens", lens ? B : 0, 4))) || (st = v.add_in(vd)) ||
        (st = v.add_in(flat(dstate_out, "dstate_out", dstate_out ? sn : 0, es))) || (st = v.add_out(vo)) ||
        (st = v.add_out(flat(dweight, "dweight", wn, 4))) ||
        (st = v.add_out(flat(dbias, "dbias", dbias ? C : 0, 4))) ||
        (st = v.add_out(flat(dstate, "dstate", dstate ? sn : 0, es))))
        return st;
    if (workspace_bytes < need) return fail(TTT_E_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if ((st = v.add_out(flat(workspace, "workspace", static_cast<int64_t>(need / 4), 4))) || (st = v.alias())) return st;
    if (!C) return ok();
    ttt::ConvBwdArgs g{{B, L, C, K, io, act == TTT_ACT_SILU, x, vx.sb, vx.st, weight, bias, state, lens,
                        nullptr, 0, 0, nullptr},
                       dy, vd.sb, vd.st, dstate_out, dx, vo.sb, vo.st, dweight, dbias, dstate,
                       static_cast<float *>(workspace)};
    return launched(ttt::launch_conv_backward(g, stream));
}

}  // extern "C"

namespace {

// sizes and options of ttt_block_norm and its backward; the gate's view
int norm_common(int B, int L, int D, int io, int resid_io, int layer, int gate_shape, int gate_act, float eps,
                const void *gate, const int64_t *gate_strides, View *vg) {
    int st;
    if ((st = check_sizes(B, L, io)) || (st = check_eps(eps))) return st;
    if (resid_io != TTT_F32 && resid_io != io)
        return fail(TTT_E_DTYPE, "resid dtype %d is neither TTT_F32 nor that of y", resid_io);
    if (D < 1 || D > TTT_NORM_MAX_D) return fail(TTT_E_SHAPE, "D = %d not in [1, %d]", D, TTT_NORM_MAX_D);
    if (layer != 0 && layer != 1) return fail(TTT_E_SHAPE, "layer = %d is not 0 / 1", layer);
    if (gate_act < TTT_ACT_NONE || gate_act > TTT_ACT_TANH)
        return fail(TTT_E_SHAPE, "gate_act = %d is not a TTT_ACT_* value", gate_act);
    if (gate_shape < TTT_GATE_NONE || gate_shape > TTT_GATE_TOKEN)
        return fail(TTT_E_SHAPE, "gate_shape = %d is not a TTT_GATE_* value", gate_shape);
    if (static_cast<int64_t>(B) * L > TTT_MAX_L) return fail(TTT_E_SHAPE, "B*L exceeds TTT_MAX_L");
    if (gate_shape == TTT_GATE_SEQUENCE && B > MAX_GRID_YZ)
        return fail(TTT_E_SHAPE, "B = %d exceeds %d with a gate for each sequence", B, MAX_GRID_YZ);
    switch (gate_shape) {
        case TTT_GATE_CHANNEL: *vg = flat(gate, "gate", D, 4); break;
        case TTT_GATE_SEQUENCE: *vg = view(gate, "gate", B, 1, 1, D, nullptr, 0, 4); break;
        case TTT_GATE_TOKEN: *vg = view(gate, "gate", B, L, 1, D, gate_strides, 2, esize(io)); break;
        default: *vg = flat(nullptr, "gate", 0, 4);
    }
    return TTT_OK;
}

}  // namespace

extern "C" {

int ttt_block_norm(int B, int L, int D, int io, int resid_io, int layer, int gate_shape, int gate_act, float eps,
                   const void *resid, const int64_t *resid_strides, const void *y, const int64_t *y_strides,
                   const void *gate, const int64_t *gate_strides, const float *post_gamma, const float *post_beta,
                   const float *pre_gamma, const float *pre_beta, const float *scale, const int *lens,
                   void *resid_out, void *x, hipStream_t stream) {
    int st;
    View vg;
    if ((st = norm_common(B, L, D, io, resid_io, layer, gate_shape, gate_act, eps, gate, gate_strides, &vg))) return st;
    const unsigned es = esize(io), rs = esize(resid_io);
    const View vr = view(resid, "resid", B, L, 1, D, resid_strides, 2, rs), vy = view(y, "y", B, L, 1, D, y_strides, 2, es);
    Views v;
    if ((st = v.add_in(vr)) || (st = v.add_in(vy)) || (st = v.add_in(vg)) ||
        (st = v.add_in(flat(post_gamma, "post_gamma", post_gamma ? D : 0, 4))) ||
        (st = v.add_in(flat(post_beta, "post_beta", post_beta ? D : 0, 4))) ||
        (st = v.add_in(flat(pre_gamma, "pre_gamma", pre_gamma ? D : 0, 4))) ||
        (st = v.add_in(flat(pre_beta, "pre_beta", pre_beta ? D : 0, 4))) ||
        (st = v.add_in(flat(scale, "scale", scale ? D : 0, 4))) ||
        (st = v.add_in(flat(lens, "lens", lens ? B : 0, 4))) ||
        (st = v.add_out(view(resid_out, "resid_out", B, L, 1, D, nullptr, 0, rs))) ||
        (st = v.add_out(view(x, "x", B, L, 1, D, nullptr, 0, es))) || (st = v.alias()))
        return st;
    if (!B || !L) return ok();
    ttt::NormArgs a{B, L, D, io, resid_io, layer, gate_act, gate_shape, eps, resid, vr.sb, vr.st, y, vy.sb, vy.st,
                    gate, gate_shape == TTT_GATE_TOKEN ? vg.sb : 0, gate_shape == TTT_GATE_TOKEN ? vg.st : 0,
                    post_gamma, post_beta, pre_gamma, pre_beta, scale, lens, resid_out, x};
    return launched(ttt::launch_block_norm(a, stream));
}

int ttt_block_norm_backward_workspace(int B, int L, int D, int gate_shape, size_t *bytes) {
    int st;
    View vg;
    if ((st = norm_common(B, L, D, TTT_F32, TTT_F32, 0, gate_shape, 0, 1e-6f, nullptr, nullptr, &vg))) return st;
    if (!bytes) return fail(TTT_E_NULL, "bytes is NULL");
    int64_t groups;
    int nq;
    ttt::block_norm_backward_partials(B, L, D, gate_shape, &groups, &nq);
    *bytes = static_cast<size_t>(groups) * nq * static_cast<size_t>(D) * sizeof(float);
    return ok();
}

int ttt_block_norm_backward(int B, int L, int D, int io, int resid_io, int layer, int gate_shape, int gate_act,
                            float eps, const void *resid, const int64_t *resid_strides, const void *y,
                            const int64_t *y_strides, const void *gate, const int64_t *gate_strides,
                            const float *post_gamma, const float *post_beta, const float *pre_gamma,
                            const float *pre_beta, const float *scale, const int *lens, const void *dresid_out,
                            const void *dx, void *dresid, void *dy, void *dgate, float *dpost_gamma,
                            float *dpost_beta, float *dpre_gamma, float *dpre_beta, float *dscale, void *workspace,
                            size_t workspace_bytes, hipStream_t stream) {
    int st;
    View vg;
    size_t need;
    if ((st = norm_common(B, L, D, io, resid_io, layer, gate_shape, gate_act, eps, gate, gate_strides, &vg)) ||
        (st = ttt_block_norm_backward_workspace(B, L, D, gate_shape, &need)))
        return st;
    const unsigned es = esize(io), rs = esize(resid_io);
    const View vr = view(resid, "resid", B, L, 1, D, resid_strides, 2, rs), vy = view(y, "y", B, L, 1, D, y_strides, 2, es);
    View vdg = vg;
    vdg.p = gate_shape == TTT_GATE_NONE ? nullptr : dgate;
    vdg.name = "dgate";
    if (gate_shape == TTT_GATE_TOKEN) vdg = view(dgate, "dgate", B, L, 1, D, nullptr, 0, es);
    Views v;
    if ((st = v.add_in(vr)) || (st = v.add_in(vy)) || (st = v.add_in(vg)) ||
        (st = v.add_in(flat(post_gamma, "post_gamma", post_gamma ? D : 0, 4))) ||
        (st = v.add_in(flat(post_beta, "post_beta", post_beta ? D : 0, 4))) ||
        (st = v.add_in(flat(pre_gamma, "pre_gamma", pre_gamma ? D : 0, 4))) ||
        (st = v.add_in(flat(scale, "scale", scale ? D : 0, 4))) ||
        (st = v.add_in(flat(lens, "lens", lens ? B : 0, 4))) ||
        (st = v.add_in(view(dresid_out, "dresid_out", B, L, 1, D, nullptr, 0, rs))) ||
        (st = v.add_in(view(dx, "dx", B, L, 1, D, nullptr, 0, es))) ||
        (st = v.add_out(view(dresid, "dresid", B, L, 1, D, nullptr, 0, rs))) ||
        (st = v.add_out(view(dy, "dy", B, L, 1, D, nullptr, 0, es))) || (st = v.add_out(vdg)) ||
        (st = v.add_out(flat(dpost_gamma, "dpost_gamma", dpost_gamma ? D : 0, 4))) ||
        (st = v.add_out(flat(dpost_beta, "dpost_beta", dpost_beta ? D : 0, 4))) ||
        (st = v.add_out(flat(dpre_gamma, "dpre_gamma", dpre_gamma ? D : 0, 4))) ||
        (st = v.add_out(flat(dpre_beta, "dpre_beta", dpre_beta ? D : 0, 4))) ||
        (st = v.add_out(flat(dscale, "dscale", dscale ? D : 0, 4))))
        return st;
    if (workspace_bytes < need) return fail(TTT_E_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if ((st = v.add_out(flat(workspace, "workspace", static_cast<int64_t>(need / 4), 4))) || (st = v.alias())) return st;
    if (!B && gate_shape == TTT_GATE_SEQUENCE) {  // no row and no gate: the other sums are zero all the same
        gate_shape = TTT_GATE_NONE;
    }
    ttt::NormBwdArgs g{{B, L, D, io, resid_io, layer, gate_act, gate_shape, eps, resid, vr.sb, vr.st, y, vy.sb, vy.st,
                        gate, gate_shape == TTT_GATE_TOKEN ? vg.sb : 0, gate_shape == TTT_GATE_TOKEN ? vg.st : 0,
                        post_gamma, post_beta, pre_gamma, pre_beta, scale, lens, nullptr, nullptr},
                       dresid_out, dx, dresid, dy, dgate, dpost_gamma, dpost_beta, dpre_gamma, dpre_beta, dscale,
                       static_cast<float *>(workspace)};
    return launched(ttt::launch_block_norm_backward(g, stream));
}

}  // extern "C"

namespace {

int ssm_common(int B, int L, int H, int P, int G, int N, int io) {
    int st;
    if ((st = check_sizes(B, L, io))) return st;
    if (P < 1 || P > TTT_SSM_MAX_DIM || N < 1 || N > TTT_SSM_MAX_DIM)
        return fail(TTT_E_SHAPE, "P = %d or N = %d not in [1, %d]", P, N, TTT_SSM_MAX_DIM);
    if (H < 1 || G < 1 || H % G) return fail(TTT_E_SHAPE, "H = %d is not a positive multiple of G = %d", H, G);
    if (static_cast<int64_t>(B) * H > TTT_SSM_MAX_HEADS)
        return fail(TTT_E_SHAPE, "B*H exceeds %d", TTT_SSM_MAX_HEADS);
    return TTT_OK;
}

// a grid's workgroups and its threads (up to 512 a workgroup) are counted in 32 bits
int ssm_plan(int B, int L, int H, int P, int N) {
    if (static_cast<int64_t>(B) * H * ((static_cast<int64_t>(L) + 63) / 64) > TTT_SSM_MAX_HEADS)
        return fail(TTT_E_SHAPE, "B*H*ceil(L/64) exceeds %d (B = %d, H = %d, L = %d)", TTT_SSM_MAX_HEADS, B, H, L);
    return TTT_OK;
}

ttt::SsmOperand operand(const View &v) { return {v.p, v.sb, v.st, v.sh}; }

// strides of a single token's operand: batch and head
View token_view(const void *p, const char *name, int64_t nb, int64_t nh, int64_t inner, const int64_t *strides,
                unsigned es) {
    View v = view(p, name, nb, 1, nh, inner, nullptr, 0, es);
    if (strides) {
        v.sb = strides[0];
        v.sh = strides[1];
    }
    return v;
}

}  // namespace

extern "C" {

int ttt_ssm_forward_workspace(int B, int L, int H, int P, int G, int N, size_t *bytes) {
    int st, nseg, seglen;
    if ((st = ssm_common(B, L, H, P, G, N, TTT_F32)) || (st = ssm_plan(B, L, H, P, N))) return st;
    if (!bytes) return fail(TTT_E_NULL, "bytes is NULL");
    // either path's segments: which one runs goes by the operands' addresses
    size_t most = 0;
    for (int mfma = 0; mfma < 2; ++mfma) {
        ttt::ssm_segments(B, L, H, N, mfma != 0, false, &nseg, &seglen);
        most = std::max(most, ttt::ssm_forward_floats(B, L, H, P, N, nseg));
    }
    *bytes = most * sizeof(float);
    return ok();
}

int ttt_ssm_forward(int B, int L, int H, int P, int G, int N, int io, const void *x, const int64_t *x_strides,
                    const void *dt, const int64_t *dt_strides, const float *A, const void *Bm,
                    const int64_t *B_strides, const void *Cm, const int64_t *C_strides, const float *D,
                    const float *dt_bias, const float *state, const int *lens, void *y, const int64_t *y_strides,
                    float *state_out, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    int st;
    size_t need;
    if ((st = ssm_common(B, L, H, P, G, N, io)) || (st = ttt_ssm_forward_workspace(B, L, H, P, G, N, &need)))
        return st;
    const unsigned es = esize(io);
    const View vx = view(x, "x", B, L, H, P, x_strides, 3, es), vt = view(dt, "dt", B, L, H, 1, dt_strides, 3, es),
               vb = view(Bm, "B", B, L, G, N, B_strides, 3, es), vc = view(Cm, "C", B, L, G, N, C_strides, 3, es),
               vy = view(y, "y", B, L, H, P, y_strides, 3, es);
    const int64_t sn = static_cast<int64_t>(B) * H * N * P;
    Views v;
    if ((st = v.add_in(vx)) || (st = v.add_in(vt)) || (st = v.add_in(flat(A, "A", H, 4))) || (st = v.add_in(vb)) ||
        (st = v.add_in(vc)) || (st = v.add_in(flat(D, "D", D ? H : 0, 4))) ||
        (st = v.add_in(flat(dt_bias, "dt_bias", dt_bias ? H : 0, 4))) ||
        (st = v.add_in(flat(state, "state", state ? sn : 0, 4))) ||
        (st = v.add_in(flat(lens, "lens", lens ? B : 0, 4))) || (st = v.add_out(vy)) ||
        (st = v.add_out(flat(state_out, "state_out", state_out ? sn : 0, 4))))
        return st;
    if (workspace_bytes < need) return fail(TTT_E_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if ((st = v.add_out(flat(workspace, "workspace", static_cast<int64_t>(need / 4), 4))) ||
        (st = v.alias(state_out, state)))
        return st;
    if (!B) return ok();
    ttt::SsmArgs a{B, L, H, P, G, N, io, operand(vx), operand(vt), operand(vb), operand(vc), A, D, dt_bias, state,
                   lens, operand(vy), state_out, static_cast<float *>(workspace), 1, 64};
    ttt::ssm_segments(B, L, H, N, ttt::ssm_mfma_supported(a), false, &a.nseg, &a.seglen);
    return launched(ttt::launch_ssm_forward(a, stream));
}

int ttt_ssm_step(int B, int H, int P, int G, int N, int io, const void *x, const int64_t *x_strides, const void *dt,
                 const int64_t *dt_strides, const float *A, const void *Bm, const int64_t *B_strides, const void *Cm,
                 const int64_t *C_strides, const float *D, const float *dt_bias, float *state, void *y,
                 hipStream_t stream) {
    int st;
    if ((st = ssm_common(B, 1, H, P, G, N, io))) return st;
    const unsigned es = esize(io);
    const View vx = token_view(x, "x", B, H, P, x_strides, es), vt = token_view(dt, "dt", B, H, 1, dt_strides, es),
               vb = token_view(Bm, "B", B, G, N, B_strides, es), vc = token_view(Cm, "C", B, G, N, C_strides, es),
               vy = token_view(y, "y", B, H, P, nullptr, es);
    const int64_t sn = static_cast<int64_t>(B) * H * N * P;
    Views v;
    if ((st = v.add_in(vx)) || (st = v.add_in(vt)) || (st = v.add_in(flat(A, "A", H, 4))) || (st = v.add_in(vb)) ||
        (st = v.add_in(vc)) || (st = v.add_in(flat(D, "D", D ? H : 0, 4))) ||
        (st = v.add_in(flat(dt_bias, "dt_bias", dt_bias ? H : 0, 4))) ||
        (st = v.add_out(flat(state, "state", sn, 4))) || (st = v.add_out(vy)) || (st = v.alias()))
        return st;
    if (!B) return ok();
    ttt::SsmArgs a{B, 1, H, P, G, N, io, operand(vx), operand(vt), operand(vb), operand(vc), A, D, dt_bias, nullptr,
                   nullptr, operand(vy), state, nullptr, 1, 64};
    return launched(ttt::launch_ssm_step(a, stream));
}

int ttt_ssm_backward_workspace(int B, int L, int H, int P, int G, int N, size_t *bytes) {
    int st, nseg, seglen;
    if ((st = ssm_common(B, L, H, P, G, N, TTT_F32)) || (st = ssm_plan(B, L, H, P, N))) return st;
    if (!bytes) return fail(TTT_E_NULL, "bytes is NULL");
    // the walks' segments, which are the shorter: the call takes them or the sweeps'
    ttt::ssm_segments(B, L, H, N, false, true, &nseg, &seglen);
    *bytes = ttt::ssm_backward_floats(B, L, H, P, N, nseg) * sizeof(float);
    return ok();
}

int ttt_ssm_backward(int B, int L, int H, int P, int G, int N, int io, const void *x, const int64_t *x_strides,
                     const void *dt, const int64_t *dt_strides, const float *A, const void *Bm,
                     const int64_t *B_strides, const void *Cm, const int64_t *C_strides, const float *D,
                     const float *dt_bias, const float *state, const int *lens, const void *dy,
                     const int64_t *dy_strides, const float *dstate_out, void *dx, const int64_t *dx_strides,
                     void *ddt, const int64_t *ddt_strides, float *dA, void *dB, const int64_t *dB_strides, void *dC,
                     const int64_t *dC_strides, float *dD, float *ddt_bias, float *dstate, void *workspace,
                     size_t workspace_bytes, hipStream_t stream) {
    int st;
    size_t need;
    if ((st = ssm_common(B, L, H, P, G, N, io)) || (st = ttt_ssm_backward_workspace(B, L, H, P, G, N, &need)))
        return st;
    const int64_t sn = static_cast<int64_t>(B) * H * N * P;
    if ((dD != nullptr) != (D != nullptr)) return fail(TTT_E_NULL, "dD is given exactly when D is");
    if ((ddt_bias != nullptr) != (dt_bias != nullptr)) return fail(TTT_E_NULL, "ddt_bias is given exactly when dt_bias is");
    if ((dstate != nullptr) != (state != nullptr) && sn) return fail(TTT_E_NULL, "dstate is given exactly when state is");
    const unsigned es = esize(io);
    const View vx = view(x, "x", B, L, H, P, x_strides, 3, es), vt = view(dt, "dt", B, L, H, 1, dt_strides, 3, es),
               vb = view(Bm, "B", B, L, G, N, B_strides, 3, es), vc = view(Cm, "C", B, L, G, N, C_strides, 3, es),
               vdy = view(dy, "dy", B, L, H, P, dy_strides, 3, es), vdx = view(dx, "dx", B, L, H, P, dx_strides, 3, es),
               vdt = view(ddt, "ddt", B, L, H, 1, ddt_strides, 3, es),
               vdb = view(dB, "dB", B, L, G, N, dB_strides, 3, es), vdc = view(dC, "dC", B, L, G, N, dC_strides, 3, es);
    Views v;
    if ((st = v.add_in(vx)) || (st = v.add_in(vt)) || (st = v.add_in(flat(A, "A", H, 4))) || (st = v.add_in(vb)) ||
        (st = v.add_in(vc)) || (st = v.add_in(flat(D, "D", D ? H : 0, 4))) ||
        (st = v.add_in(flat(dt_bias, "dt_bias", dt_bias ? H : 0, 4))) ||
        (st = v.add_in(flat(state, "state", state ? sn : 0, 4))) ||
        (st = v.add_in(flat(lens, "lens", lens ? B : 0, 4))) || (st = v.add_in(vdy)) ||
        (st = v.add_in(flat(dstate_out, "dstate_out", dstate_out ? sn : 0, 4))) || (st = v.add_out(vdx)) ||
        (st = v.add_out(vdt)) || (st = v.add_out(flat(dA, "dA", H, 4))) || (st = v.add_out(vdb)) ||
        (st = v.add_out(vdc)) || (st = v.add_out(flat(dD, "dD", dD ? H : 0, 4))) ||
        (st = v.add_out(flat(ddt_bias, "ddt_bias", ddt_bias ? H : 0, 4))) ||
        (st = v.add_out(flat(dstate, "dstate", dstate ? sn : 0, 4))))
        return st;
    if (workspace_bytes < need) return fail(TTT_E_SHAPE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if ((st = v.add_out(flat(workspace, "workspace", static_cast<int64_t>(need / 4), 4))) || (st = v.alias())) return st;
    ttt::SsmBwdArgs g{{B, L, H, P, G, N, io, operand(vx), operand(vt), operand(vb), operand(vc), A, D, dt_bias,
                       state, lens, {nullptr, 0, 0, 0}, nullptr, static_cast<float *>(workspace), 1, 64},
                      operand(vdy), dstate_out, operand(vdx), operand(vdt), operand(vdb), operand(vdc), dA, dD,
                      ddt_bias, dstate};
    ttt::ssm_segments(B, L, H, N, ttt::ssm_bwd_mfma_supported(g), true, &g.f.nseg, &g.f.seglen);
    return launched(ttt::launch_ssm_backward(g, stream));
}

}  // extern "C"
