// Strided operands of the operators around the layer, as their extern "C"
// entry points check them on the host.
#pragma once

#include <algorithm>
#include <utility>

#include "abi_common.hpp"

namespace ttt {
namespace abi {

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
inline View view(const void *p, const char *name, int64_t nb, int64_t nt, int64_t nh, int64_t inner,
          const int64_t *strides, int rank, unsigned es) {
    View v{p, name, nb, nt, nh, inner, nt * nh * inner, nh * inner, inner, es};
    if (strides) {
        v.sb = strides[0];
        if (rank > 1) v.st = strides[1];
        if (rank > 2) v.sh = strides[2];
    }
    return v;
}

inline bool empty(const View &v) { return !v.nb || !v.nt || !v.nh || !v.inner; }

// bytes from the first to behind the last element; false on overflow
inline bool extent(const View &v, size_t *out) {
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

inline int check_view(const View &v, bool out, size_t *bytes) {
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
inline bool apart(const View &a, const View &b) {
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

inline View flat(const void *p, const char *name, int64_t n, unsigned es) {
    return view(p, name, 1, 1, 1, n, nullptr, 0, es);
}

inline int check_sizes(int B, int L, int io) {
    if (B < 0 || L < 0) return fail(TTT_E_SHAPE, "negative size (B=%d L=%d)", B, L);
    if (io != TTT_F32 && io != TTT_BF16) return fail(TTT_E_DTYPE, "io dtype %d is not TTT_F32/TTT_BF16", io);
    if (L > TTT_MAX_L) return fail(TTT_E_SHAPE, "L = %d exceeds TTT_MAX_L = %d", L, TTT_MAX_L);
    return TTT_OK;
}

constexpr int MAX_GRID_YZ = 65535;

inline unsigned esize(int io) { return io == TTT_BF16 ? 2 : 4; }

}  // namespace abi
}  // namespace ttt
