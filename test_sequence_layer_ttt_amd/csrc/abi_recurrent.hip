// extern "C" entry points of the gated linear recurrence and the 8-bit integer
// product (declared and documented in ttt.h): validation on the host, then the
// launch. Nothing here allocates or synchronises.
#include "abi_view.hpp"
#include "i8.hpp"
#include "lru.hpp"

using namespace ttt::abi;

namespace {

int lru_common(int B, int L, int D, int io) {
    int st;
    if ((st = check_sizes(B, L, io))) return st;
    if (D < 1 || D > TTT_LRU_MAX_D) return fail(TTT_E_SHAPE, "D = %d not in [1, %d]", D, TTT_LRU_MAX_D);
    if (B > MAX_GRID_YZ) return fail(TTT_E_SHAPE, "B = %d exceeds %d", B, MAX_GRID_YZ);
    // tiles of 64 tokens: a grid's workgroups and threads are counted in 32 bits
    if (static_cast<int64_t>(B > 1 ? B : 1) * ((static_cast<int64_t>(L) + 63) / 64) > TTT_LRU_MAX_TILES)
        return fail(TTT_E_SHAPE, "B*ceil(L/64) exceeds %d (B = %d, L = %d)", TTT_LRU_MAX_TILES, B, L);
    if (L > 64 && B * ((static_cast<int64_t>(L) + 63) / 64) * ((D + 127) / 128) >= 1 << 24)
        return fail(TTT_E_SHAPE, "B*ceil(L/64)*ceil(D/128) is 2^24 or more (B = %d, L = %d, D = %d)", B, L, D);
    return TTT_OK;
}

View optional(const void *p, const char *name, int B, int L, int D, const int64_t *strides, unsigned es) {
    return p ? view(p, name, B, L, 1, D, strides, 2, es) : flat(nullptr, name, 0, es);
}

int scratch(const void *workspace, size_t bytes, size_t need) {
    if (bytes < need) return fail(TTT_E_SHAPE, "workspace of %zu bytes, %zu needed", bytes, need);
    if (need && (reinterpret_cast<uintptr_t>(workspace) & 15))
        return fail(TTT_E_ALIGN, "workspace (%p) is not 16-byte aligned", workspace);
    return TTT_OK;
}

}  // namespace

extern "C" {

int ttt_lru_forward_workspace(int B, int L, int D, size_t *bytes) {
    int st;
    if ((st = lru_common(B, L, D, TTT_F32))) return st;
    if (!bytes) return fail(TTT_E_NULL, "bytes is NULL");
    *bytes = static_cast<size_t>(ttt::lru_forward_floats(B, L, D)) * sizeof(float);
    return ok();
}

int ttt_lru_forward(int B, int L, int D, int io, const void *x, const int64_t *x_strides, const void *r,
                    const int64_t *r_strides, const void *i, const int64_t *i_strides, const float *rate,
                    const float *state, const int *lens, void *y, const int64_t *y_strides, float *state_out,
                    void *workspace, size_t workspace_bytes, hipStream_t stream) {
    int st;
    size_t need;
    if ((st = lru_common(B, L, D, io)) || (st = ttt_lru_forward_workspace(B, L, D, &need))) return st;
    const unsigned es = esize(io);
    const int64_t sn = static_cast<int64_t>(B) * D;
    const View vx = view(x, "x", B, L, 1, D, x_strides, 2, es), vr = view(r, "r", B, L, 1, D, r_strides, 2, es),
               vi = optional(i, "i", B, L, D, i_strides, es), vy = view(y, "y", B, L, 1, D, y_strides, 2, es);
    Views v;
    if ((st = v.add_in(vx)) || (st = v.add_in(vr)) || (st = v.add_in(vi)) ||
        (st = v.add_in(flat(rate, "rate", rate ? D : 0, 4))) || (st = v.add_in(flat(state, "state", state ? sn : 0, 4))) ||
        (st = v.add_in(flat(lens, "lens", lens ? B : 0, 4))) || (st = v.add_out(vy)) ||
        (st = v.add_out(flat(state_out, "state_out", state_out ? sn : 0, 4))))
        return st;
    if ((st = scratch(workspace, workspace_bytes, need)) ||
        (st = v.add_out(flat(workspace, "workspace", static_cast<int64_t>(need / 4), 4))) ||
        (st = v.alias(state_out, state)))
        return st;
    if (!B || (!L && !state_out)) return ok();
    ttt::LruArgs a{B, L, D, io, x, r, i, vx.sb, vx.st, vr.sb, vr.st, vi.sb, vi.st, rate, state, lens,
                   y, vy.sb, vy.st, state_out, static_cast<float *>(workspace)};
    return launched(ttt::launch_lru_forward(a, stream));
}

int ttt_lru_step(int B, int D, int io, const void *x, const int64_t *x_strides, const void *r, const int64_t *r_strides,
                 const void *i, const int64_t *i_strides, const float *rate, float *state, void *y,
                 hipStream_t stream) {
    int st;
    if ((st = check_sizes(B, 1, io))) return st;
    if (D < 1 || D > TTT_LRU_MAX_D) return fail(TTT_E_SHAPE, "D = %d not in [1, %d]", D, TTT_LRU_MAX_D);
    if (static_cast<int64_t>(B) * D > INT_MAX) return fail(TTT_E_SHAPE, "B*D too large");
    const unsigned es = esize(io);
    const View vx = view(x, "x", B, 1, 1, D, x_strides, 1, es), vr = view(r, "r", B, 1, 1, D, r_strides, 1, es),
               vi = i ? view(i, "i", B, 1, 1, D, i_strides, 1, es) : flat(nullptr, "i", 0, es),
               vy = view(y, "y", B, 1, 1, D, nullptr, 0, es);
    Views v;
    if ((st = v.add_in(vx)) || (st = v.add_in(vr)) || (st = v.add_in(vi)) ||
        (st = v.add_in(flat(rate, "rate", rate ? D : 0, 4))) ||
        (st = v.add_out(flat(state, "state", static_cast<int64_t>(B) * D, 4))) || (st = v.add_out(vy)) || (st = v.alias()))
        return st;
    if (!B) return ok();
    ttt::LruArgs a{B, 1, D, io, x, r, i, vx.sb, vx.st, vr.sb, vr.st, vi.sb, vi.st, rate, nullptr, nullptr,
                   y, vy.sb, vy.st, state, nullptr};
    return launched(ttt::launch_lru_step(a, stream));
}

int ttt_lru_backward_workspace(int B, int L, int D, size_t *bytes) {
    int st;
    if ((st = lru_common(B, L, D, TTT_F32))) return st;
    if (!bytes) return fail(TTT_E_NULL, "bytes is NULL");
    *bytes = static_cast<size_t>(ttt::lru_backward_floats(B, L, D)) * sizeof(float);
    return ok();
}

int ttt_lru_backward(int B, int L, int D, int io, const void *x, const int64_t *x_strides, const void *r,
                     const int64_t *r_strides, const void *i, const int64_t *i_strides, const float *rate,
                     const float *state, const int *lens, const void *dy, const int64_t *dy_strides,
                     const float *dstate_out, void *dx, const int64_t *dx_strides, void *dr,
                     const int64_t *dr_strides, void *di, const int64_t *di_strides, float *drate, float *dstate,
                     void *workspace, size_t workspace_bytes, hipStream_t stream) {
    int st;
    size_t need;
    if ((st = lru_common(B, L, D, io)) || (st = ttt_lru_backward_workspace(B, L, D, &need))) return st;
    const unsigned es = esize(io);
    const int64_t sn = static_cast<int64_t>(B) * D;
    if ((di != nullptr) != (i != nullptr) && sn && L) return fail(TTT_E_NULL, "di is given exactly when i is");
    if ((drate != nullptr) != (rate != nullptr)) return fail(TTT_E_NULL, "drate is given exactly when rate is");
    if ((dstate != nullptr) != (state != nullptr) && sn) return fail(TTT_E_NULL, "dstate is given exactly when state is");
    const View vx = view(x, "x", B, L, 1, D, x_strides, 2, es), vr = view(r, "r", B, L, 1, D, r_strides, 2, es),
               vi = optional(i, "i", B, L, D, i_strides, es), vd = view(dy, "dy", B, L, 1, D, dy_strides, 2, es),
               vdx = view(dx, "dx", B, L, 1, D, dx_strides, 2, es), vdr = view(dr, "dr", B, L, 1, D, dr_strides, 2, es),
               vdi = optional(di, "di", B, L, D, di_strides, es);
    Views v;
    if ((st = v.add_in(vx)) || (st = v.add_in(vr)) || (st = v.add_in(vi)) ||
        (st = v.add_in(flat(rate, "rate", rate ? D : 0, 4))) || (st = v.add_in(flat(state, "state", state ? sn : 0, 4))) ||
        (st = v.add_in(flat(lens, "lens", lens ? B : 0, 4))) || (st = v.add_in(vd)) ||
        (st = v.add_in(flat(dstate_out, "dstate_out", dstate_out ? sn : 0, 4))) || (st = v.add_out(vdx)) ||
        (st = v.add_out(vdr)) || (st = v.add_out(vdi)) || (st = v.add_out(flat(drate, "drate", drate ? D : 0, 4))) ||
        (st = v.add_out(flat(dstate, "dstate", dstate ? sn : 0, 4))))
        return st;
    if ((st = scratch(workspace, workspace_bytes, need)) ||
        (st = v.add_out(flat(workspace, "workspace", static_cast<int64_t>(need / 4), 4))) || (st = v.alias())) return st;
    ttt::LruBwdArgs g{{B, L, D, io, x, r, i, vx.sb, vx.st, vr.sb, vr.st, vi.sb, vi.st, rate, state, lens, nullptr, 0, 0,
                       nullptr, static_cast<float *>(workspace)},
                      dy, vd.sb, vd.st, dstate_out, dx, dr, di, vdx.sb, vdx.st, vdr.sb, vdr.st, vdi.sb, vdi.st, drate, dstate};
    return launched(ttt::launch_lru_backward(g, stream));
}

}  // extern "C"

namespace {

int i8_sizes(int M, int K, int N) {
    if (M < 0 || N < 0) return fail(TTT_E_SHAPE, "negative size (M=%d N=%d)", M, N);
    if (K < 1 || K > TTT_I8_MAX_K) return fail(TTT_E_SHAPE, "K = %d not in [1, %d]", K, TTT_I8_MAX_K);
    if (M > TTT_I8_MAX_ROWS || N > TTT_I8_MAX_ROWS)
        return fail(TTT_E_SHAPE, "M = %d or N = %d exceeds %d", M, N, TTT_I8_MAX_ROWS);
    // tiles of 64 x 64: a grid's workgroups and threads are counted in 32 bits
    if (((static_cast<int64_t>(M) + 63) / 64) * ((static_cast<int64_t>(N) + 63) / 64) > TTT_I8_MAX_TILES)
        return fail(TTT_E_SHAPE, "ceil(M/64)*ceil(N/64) exceeds %d (M = %d, N = %d)", TTT_I8_MAX_TILES, M, N);
    return TTT_OK;
}

View rows(const void *p, const char *name, int64_t n, int64_t inner, const int64_t *strides, unsigned es) {
    return view(p, name, n, 1, 1, inner, strides, 1, es);
}

// rows in whole 128-byte lines
int64_t padded(int K) { return (static_cast<int64_t>(K) + 127) / 128 * 128; }

// The product, operands that it cannot take as they stand laid out anew in `room` (x first) before.
hipError_t project(ttt::I8Args a, bool px, bool pw, int8_t *room, hipStream_t stream) {
    const int pad = static_cast<int>(padded(a.K));
    int8_t *x = room, *w = room + (px ? static_cast<int64_t>(a.M) * pad : 0);
    if (px || pw) {
        const ttt::I8PadArgs p{{px ? a.M : 0, pw ? a.N : 0}, {a.x, a.w}, {a.xr, a.wr}, {x, w}, a.K, pad};
        const hipError_t e = ttt::launch_i8_pad(p, stream);
        if (e != hipSuccess) return e;
        if (px) a.x = x, a.xr = pad;
        if (pw) a.w = w, a.wr = pad;
        a.K = (a.K + 15) / 16 * 16;  // zeros of w, at least, behind a K that is no multiple
    }
    return ttt::launch_i8_project(a, stream);
}

// A product of features: the workspace holds the quantised rows, their scales and, where w's rows
// cannot be taken as they stand, these.
size_t features_bytes(int M, int K, int N) {
    return static_cast<size_t>(M) * padded(K) + (static_cast<size_t>(M) + 3) / 4 * 16 + static_cast<size_t>(N) * padded(K);
}
bool unaligned_w(const ttt::I8Args &a) {
    bool x, w;
    ttt::i8_unaligned(a, &x, &w);
    return w;
}
int features(int io, const void *x, int64_t xr, void *workspace, ttt::I8Args *a, hipStream_t stream) {
    if (ttt::i8_features_in_one(*a)) return launched(ttt::launch_i8_features(*a, io, x, xr, stream));
    const int64_t pad = padded(a->K);
    int8_t *q = static_cast<int8_t *>(workspace);
    float *scale = reinterpret_cast<float *>(q + a->M * pad);
    a->x = q;
    a->xr = pad;
    a->xs = scale;
    const hipError_t e = ttt::launch_i8_quantize({a->M, a->K, io, x, xr, q, pad, scale}, stream);
    // whole lines of their own: with K no multiple of 16 the bytes behind a row meet zeros of w
    return launched(e == hipSuccess ? project(*a, false, unaligned_w(*a), q + a->M * pad + (a->M + 3) / 4 * 16, stream) : e);
}

}  // namespace

extern "C" {

int ttt_i8_quantize(int M, int K, int io, const void *x, const int64_t *x_strides, int8_t *q, const int64_t *q_strides,
                    float *scale, hipStream_t stream) {
    int st;
    if ((st = i8_sizes(M, K, 0))) return st;
    if (io != TTT_F32 && io != TTT_BF16) return fail(TTT_E_DTYPE, "io dtype %d is not TTT_F32/TTT_BF16", io);
    const View vx = rows(x, "x", M, K, x_strides, esize(io)), vq = rows(q, "q", M, K, q_strides, 1);
    Views v;
    if ((st = v.add_in(vx)) || (st = v.add_out(vq)) || (st = v.add_out(flat(scale, "scale", M, 4))) || (st = v.alias()))
        return st;
    if (!M) return ok();
    return launched(ttt::launch_i8_quantize({M, K, io, x, vx.sb, q, vq.sb, scale}, stream));
}

int ttt_i8_project_workspace(int M, int K, int N, const int8_t *x, const int64_t *x_strides, const int8_t *w,
                             const int64_t *w_strides, size_t *bytes) {
    int st;
    if ((st = i8_sizes(M, K, N))) return st;
    if (!bytes) return fail(TTT_E_NULL, "bytes is NULL");
    ttt::I8Args a{M, K, N, 0, x, x_strides ? x_strides[0] : K, nullptr, w, w_strides ? w_strides[0] : K};
    bool px, pw;
    ttt::i8_unaligned(a, &px, &pw);
    *bytes = M && N ? ((px ? static_cast<size_t>(M) : 0) + (pw ? N : 0)) * padded(K) : 0;
    return ok();
}

int ttt_i8_project(int M, int K, int N, int out_io, const int8_t *x, const int64_t *x_strides, const float *x_scale,
                   const int8_t *w, const int64_t *w_strides, const float *w_scale, const float *bias, void *y,
                   const int64_t *y_strides, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    int st;
    if ((st = i8_sizes(M, K, N))) return st;
    if (out_io != TTT_F32 && out_io != TTT_BF16)
        return fail(TTT_E_DTYPE, "output dtype %d is not TTT_F32/TTT_BF16", out_io);
    const View vx = rows(x, "x", M, K, x_strides, 1), vw = rows(w, "w", N, K, w_strides, 1),
               vy = rows(y, "y", M, N, y_strides, esize(out_io));
    const ttt::I8Args a{M, K, N, out_io, x, vx.sb, x_scale, w, vw.sb, w_scale, bias, y, vy.sb};
    bool px, pw;
    ttt::i8_unaligned(a, &px, &pw);
    size_t need;
    if ((st = ttt_i8_project_workspace(M, K, N, x, x_strides, w, w_strides, &need))) return st;
    Views v;
    if ((st = v.add_in(vx)) || (st = v.add_in(flat(x_scale, "x_scale", M, 4))) || (st = v.add_in(vw)) ||
        (st = v.add_in(flat(w_scale, "w_scale", N, 4))) || (st = v.add_in(flat(bias, "bias", bias ? N : 0, 4))) ||
        (st = v.add_out(vy)) || (st = scratch(workspace, workspace_bytes, need)) ||
        (st = v.add_out(flat(need ? workspace : nullptr, "workspace", static_cast<int64_t>(need / 4), 4))) || (st = v.alias()))
        return st;
    if (!M || !N) return ok();
    return launched(project(a, px, pw, static_cast<int8_t *>(workspace), stream));
}

int ttt_i8_linear_workspace(int M, int K, int N, const int8_t *w, const int64_t *w_strides, size_t *bytes) {
    int st;
    if ((st = i8_sizes(M, K, N))) return st;
    if (!bytes) return fail(TTT_E_NULL, "bytes is NULL");
    const ttt::I8Args a{M, K, N, 0, nullptr, K, nullptr, w, w_strides ? w_strides[0] : K};
    *bytes = features_bytes(M, K, unaligned_w(a) ? N : 0);
    return ok();
}

int ttt_i8_linear(int M, int K, int N, int io, const void *x, const int64_t *x_strides, const int8_t *w,
                  const int64_t *w_strides, const float *w_scale, const float *bias, void *y, const int64_t *y_strides,
                  void *workspace, size_t workspace_bytes, hipStream_t stream) {
    int st;
    size_t need;
    if ((st = i8_sizes(M, K, N))) return st;
    if (io != TTT_F32 && io != TTT_BF16) return fail(TTT_E_DTYPE, "io dtype %d is not TTT_F32/TTT_BF16", io);
    const View vx = rows(x, "x", M, K, x_strides, esize(io)), vw = rows(w, "w", N, K, w_strides, 1),
               vy = rows(y, "y", M, N, y_strides, esize(io));
    ttt::I8Args a{M, K, N, io, nullptr, 0, nullptr, w, vw.sb, w_scale, bias, y, vy.sb};
    if ((st = ttt_i8_linear_workspace(M, K, N, w, w_strides, &need))) return st;
    Views v;
    if ((st = v.add_in(vx)) || (st = v.add_in(vw)) || (st = v.add_in(flat(w_scale, "w_scale", N, 4))) ||
        (st = v.add_in(flat(bias, "bias", bias ? N : 0, 4))) || (st = v.add_out(vy)))
        return st;
    if ((st = scratch(workspace, workspace_bytes, need)) ||
        (st = v.add_out(flat(workspace, "workspace", static_cast<int64_t>(need / 4), 4))) || (st = v.alias())) return st;
    if (!M || !N) return ok();
    return features(io, x, vx.sb, workspace, &a, stream);
}

int ttt_qkv_project_i8(int B, int L, int d_model, int H, int d, const void *X, const int8_t *theta,
                       const float *theta_scale, void *XQ, void *XK, void *XV, void *workspace, size_t workspace_bytes,
                       hipStream_t stream) {
    int st;
    if (B < 0 || L < 0 || H < 0) return fail(TTT_E_SHAPE, "negative size (B=%d L=%d H=%d)", B, L, H);
    if (d != 64) return fail(TTT_E_SHAPE, "d = %d: the projection serves d = 64", d);
    const int64_t M = static_cast<int64_t>(B) * L, N = 192 * static_cast<int64_t>(H);
    if (M > TTT_I8_MAX_ROWS || N > TTT_I8_MAX_ROWS) return fail(TTT_E_SHAPE, "B*L or 3*H*d exceeds %d", TTT_I8_MAX_ROWS);
    size_t need;
    if ((st = i8_sizes(static_cast<int>(M), d_model, static_cast<int>(N)))) return st;
    ttt::I8Args a{static_cast<int>(M), d_model, static_cast<int>(N), TTT_BF16, nullptr, 0, nullptr, theta, d_model,
                  theta_scale, nullptr, nullptr, 0, L, H, {XQ, XK, XV}};
    if ((st = ttt_i8_linear_workspace(a.M, a.K, a.N, theta, nullptr, &need))) return st;
    void *out[3] = {XQ, XK, XV};
    const char *names[3] = {"XQ", "XK", "XV"};
    Views v;
    if ((st = v.add_in(rows(X, "X", M, d_model, nullptr, 2))) || (st = v.add_in(rows(theta, "theta", N, d_model, nullptr, 1))) ||
        (st = v.add_in(flat(theta_scale, "theta_scale", N, 4))))
        return st;
    for (int k = 0; k < 3; ++k) {
        if ((st = v.add_out(flat(out[k], names[k], M * H * 64, 2)))) return st;
        if (M * H && (reinterpret_cast<uintptr_t>(out[k]) & 15))
            return fail(TTT_E_ALIGN, "%s (%p) is not 16-byte aligned", names[k], out[k]);
    }
    if ((st = scratch(workspace, workspace_bytes, need)) ||
        (st = v.add_out(flat(workspace, "workspace", static_cast<int64_t>(need / 4), 4))) || (st = v.alias())) return st;
    if (!M || !N) return ok();
    return features(TTT_BF16, X, d_model, workspace, &a, stream);
}

}  // extern "C"
