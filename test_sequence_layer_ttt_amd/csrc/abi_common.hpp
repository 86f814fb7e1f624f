// Host-side argument checks shared by the extern "C" entry points of libttt.so.
#pragma once

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <initializer_list>

#include <hip/hip_runtime.h>

#include "ttt.h"

namespace ttt {
namespace abi {

inline thread_local char g_err[512] = "";

inline int fail(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}

inline int ok() {
    g_err[0] = '\0';
    return TTT_OK;
}

struct Buf {
    const void *p;
    size_t bytes;
    const char *name;
    bool optional;
    unsigned align;  // required alignment in bytes
};

inline bool mul_ok(size_t a, size_t b, size_t *out) { return !__builtin_mul_overflow(a, b, out); }

// product of non-negative ints as bytes; false on overflow
inline bool nbytes(size_t *out, std::initializer_list<size_t> dims) {
    size_t r = 1;
    for (size_t v : dims)
        if (!mul_ok(r, v, &r)) return false;
    *out = r;
    return true;
}

inline int check_bufs(const Buf *b, int n) {
    for (int i = 0; i < n; ++i) {
        if (!b[i].p) {
            if (b[i].bytes && !b[i].optional)
                return fail(TTT_E_NULL, "%s is NULL (%zu bytes expected)", b[i].name, b[i].bytes);
            continue;
        }
        if (reinterpret_cast<uintptr_t>(b[i].p) & (b[i].align - 1))
            return fail(TTT_E_ALIGN, "%s (%p) is not %u-byte aligned", b[i].name, b[i].p, b[i].align);
    }
    return TTT_OK;
}

inline bool overlaps(const Buf &a, const Buf &b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Outputs must not overlap any other buffer, except that an output may be
// exactly the same buffer as its paired input (`same_ok[out] == in`).
inline int check_alias(const Buf *outs, int nout, const Buf *ins, int nin, const int *pair) {
    for (int o = 0; o < nout; ++o) {
        for (int i = 0; i < nin; ++i) {
            if (!overlaps(outs[o], ins[i])) continue;
            if (pair && pair[o] == i && outs[o].p == ins[i].p && outs[o].bytes == ins[i].bytes) continue;
            return fail(TTT_E_ALIAS, "%s overlaps %s", outs[o].name, ins[i].name);
        }
        for (int o2 = o + 1; o2 < nout; ++o2)
            if (overlaps(outs[o], outs[o2]))
                return fail(TTT_E_ALIAS, "%s overlaps %s", outs[o].name, outs[o2].name);
    }
    return TTT_OK;
}

inline int check_common(int B, int H, int L, int mb, int io) {
    if (B < 0 || H < 0 || L < 0) return fail(TTT_E_SHAPE, "negative size (B=%d H=%d L=%d)", B, H, L);
    if (io != TTT_F32 && io != TTT_BF16) return fail(TTT_E_DTYPE, "io dtype %d is not TTT_F32/TTT_BF16", io);
    if (mb < 1 || mb > 16) return fail(TTT_E_SHAPE, "mini-batch size %d not in [1, 16]", mb);
    // token and chunk indices inside the kernels are 32-bit ints
    if (L > TTT_MAX_L) return fail(TTT_E_SHAPE, "L = %d exceeds TTT_MAX_L = %d", L, TTT_MAX_L);
    if (static_cast<long long>(B) * H > INT_MAX) return fail(TTT_E_SHAPE, "B*H = %lld too large", static_cast<long long>(B) * H);
    return TTT_OK;
}

// The layer norms evaluate 1/sqrt(var + eps) with var >= 0, which needs a
// positive normal eps.
inline int check_eps(float eps) {
    if (!(eps >= FLT_MIN) || !std::isfinite(eps))
        return fail(TTT_E_SHAPE, "ln_eps = %g is not a positive normal float", static_cast<double>(eps));
    return TTT_OK;
}

inline int launched(hipError_t e) {
    if (e != hipSuccess) return fail(TTT_E_HIP, "kernel launch failed: %s", hipGetErrorString(e));
    return ok();
}

}  // namespace abi
}  // namespace ttt
