// Python binding of the operators around the layer (_block.so): argument
// marshalling only. It checks type, shape, layout and device of torch tensors,
// makes the outputs and workspaces that are not given, and calls libttt.so's
// C ABI on the operands' device and its current stream. A call costs 3 to 4 us,
// 2.7 of them the launch and 0.4 each output; the same checks in Python through
// ctypes cost 9 to 13 us, more than the kernels of a single token take. block.py
// documents the functions.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <string>
#include <vector>

#include "ttt.h"

namespace {

using at::Tensor;
typedef std::vector<int64_t> Shape;

struct PyError {};  // a Python exception is set

PyObject *ttt_error = nullptr;  // TTTError, set by init()

[[noreturn]] void raise(PyObject *type, const std::string &msg) {
    PyErr_SetString(type, msg.c_str());
    throw PyError{};
}

std::string text(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kInt: return "torch.int32";
        case at::kHalf: return "torch.float16";
        case at::kDouble: return "torch.float64";
        case at::kLong: return "torch.int64";
        case at::kChar: return "torch.int8";
        default: return std::string("torch.") + c10::toString(t);
    }
}
std::string text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

// the device and storage type that the operands share
struct Kind {
    int index;
    at::ScalarType dt;
    int io;
};

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

int io_of(const Tensor &t, const char *name) {
    if (t.scalar_type() == at::kBFloat16) return TTT_BF16;
    if (t.scalar_type() == at::kFloat) return TTT_F32;
    raise(PyExc_TypeError, std::string(name) + " dtype " + text(t.scalar_type()) + " not supported");
}

// a rank that the caller goes by
const Tensor &ranked(PyObject *o, const char *name, std::initializer_list<int64_t> ranks) {
    const Tensor &t = tensor(o, name);
    for (int64_t r : ranks)
        if (t.dim() == r) return t;
    raise(PyExc_ValueError, std::string(name) + " has shape " + text(t.sizes()) + ", expected " +
                                std::to_string(*ranks.begin()) + " dimensions");
}

Kind kind_of(const Tensor &t, const char *name) {
    const int io = io_of(t, name);
    if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a device tensor (got " + t.device().str() + ")");
    return {static_cast<int>(t.get_device()), t.scalar_type(), io};
}

const Tensor &check(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType dt, const Kind &k,
                    bool contiguous = true) {
    const Tensor &t = tensor(o, name);
    if (t.scalar_type() != dt)
        raise(PyExc_TypeError, std::string(name) + " has dtype " + text(t.scalar_type()) + ", expected " + text(dt));
    if (t.sizes() != shape)
        raise(PyExc_ValueError, std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(shape));
    if (!t.is_cuda() || t.get_device() != k.index)
        raise(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(k.index));
    if (contiguous && !t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t;
}

// address of a checked tensor, null where it is None (or holds nothing)
void *ptr(const Tensor &t) { return t.numel() ? t.data_ptr() : nullptr; }
template <typename T = void>
T *opt(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType dt, const Kind &k) {
    return o == Py_None ? nullptr : static_cast<T *>(ptr(check(o, name, shape, dt, k)));
}

// a strided operand: address, and the strides of all but the innermost `skip`
// dimensions (null: contiguous)
struct Operand {
    void *p;
    int64_t s[3];
    const int64_t *strides;
    Operand(const Tensor &t, const char *name, int skip = 1) : p(ptr(t)), s{}, strides(nullptr) {
        if (t.is_contiguous()) return;
        if (skip && t.size(-1) > 1 && t.stride(-1) != 1)
            raise(PyExc_ValueError, std::string("the innermost dimension of ") + name + " must be contiguous");
        for (int64_t i = 0; i < t.dim() - skip; ++i) s[i] = t.stride(i);
        strides = s;
    }
    Operand(const Operand &) = delete;
};

// straight from the caching allocator, on the device's current stream: past the
// dispatcher, which takes as long again
Tensor make(at::IntArrayRef shape, at::ScalarType dt, const Kind &k) {
    return at::detail::empty_cuda(shape, dt, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(k.index)), std::nullopt);
}
// an output: as given (checked) or new
Tensor output(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType dt, const Kind &k, bool contiguous = true) {
    return o == Py_None ? make(shape, dt, k) : check(o, name, shape, dt, k, contiguous);
}

// What a call has written into a tensor of the caller's changes its version, so
// that autograd does not go back through what it saved of it before (tensors of
// inference mode have none).
void written(const Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(PyObject *given, const Tensor &t) {  // an output that may be new
    if (given != Py_None) written(t);
}

void done(int code) {
    if (code == TTT_OK) return;
    PyObject *e = PyObject_CallFunction(ttt_error, "is", code, ttt_last_error());
    if (e) {
        PyErr_SetObject(ttt_error, e);
        Py_DECREF(e);
    }
    throw PyError{};
}

// Runs `fn(stream)` on the operands' device and its current stream.
template <typename F> void call(const Kind &k, F fn) {
    int code = 0;
    auto run = [&] {
        const hipStream_t s = c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(k.index)).stream();
        PyThreadState *ts = PyEval_SaveThread();
        code = fn(s);
        PyEval_RestoreThread(ts);
    };
    if (c10::hip::current_device() == k.index) {
        run();
    } else {
        const c10::DeviceGuard guard(at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(k.index)));
        run();
    }
    done(code);
}

struct Workspace {
    Tensor t;
    void *p = nullptr;
    size_t bytes = 0;
    Workspace(PyObject *o, size_t need, const Kind &k) {
        if (o == Py_None) {
            if (!need) return;
            t = make({static_cast<int64_t>(need)}, at::kByte, k);
        } else {
            t = tensor(o, "workspace");
            if (!t.is_cuda() || t.get_device() != k.index || !t.is_contiguous())
                raise(PyExc_ValueError, "workspace must be a contiguous tensor on the operands' device");
        }
        p = ptr(t);
        bytes = t.numel() * t.element_size();
    }
};

// The gradients of a backward: from the dict that is given, or new ones.
struct Grads {
    PyObject *given, *dict;
    const Kind &k;
    Py_ssize_t n = 0;
    Grads(PyObject *g, const Kind &kind) : given(g), dict(nullptr), k(kind) {
        if (given == Py_None) {
            dict = PyDict_New();
            if (!dict) throw PyError{};
        } else if (!PyDict_Check(given)) {
            raise(PyExc_ValueError, "grads must be a dict of outputs");
        }
    }
    ~Grads() { Py_XDECREF(dict); }
    Tensor get(const char *name, at::IntArrayRef shape, at::ScalarType dt, bool contiguous = true) {
        ++n;
        if (dict) {
            const Tensor t = make(shape, dt, k);
            PyObject *o = THPVariable_Wrap(t);
            const int bad = o ? PyDict_SetItemString(dict, name, o) : -1;
            Py_XDECREF(o);
            if (bad) throw PyError{};
            return t;
        }
        PyObject *o = PyDict_GetItemString(given, name);
        if (!o) raise(PyExc_ValueError, std::string("grads has no ") + name);
        return check(o, name, shape, dt, k, contiguous);
    }
    // every name that is expected was asked for: none may be left over
    void whole() const {
        if (!dict && PyDict_Size(given) != n) raise(PyExc_ValueError, "grads has outputs that this call does not make");
    }
    PyObject *take() {
        PyObject *r = dict ? dict : given;
        if (!dict) {
            PyObject *key, *value;
            for (Py_ssize_t i = 0; PyDict_Next(given, &i, &key, &value);)
                if (THPVariable_Check(value)) written(THPVariable_Unpack(value));  // others ran since it was checked
            Py_INCREF(r);
        }
        dict = nullptr;
        return r;
    }
};

PyObject *pair(const Tensor &a, const Tensor &b) {
    PyObject *x = THPVariable_Wrap(a), *y = THPVariable_Wrap(b);
    PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

int number(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw PyError{};
    return static_cast<int>(v);
}

int size(int64_t n, const char *what) {  // the ABI's sizes are ints
    if (n > INT32_MAX) raise(PyExc_ValueError, std::string(what) + " = " + std::to_string(n) + " is too large");
    return static_cast<int>(n);
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N> PyObject *method(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(a);
    } catch (const PyError &) {
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// --- convolution ---------------------------------------------------------------

struct ConvIn {
    const Tensor &x;
    Kind k;
    int B, L, C, K;
    const float *w, *bias;
    ConvIn(PyObject *ox, PyObject *ow, PyObject *ob, bool one)
        : x(ranked(ox, "x", {one ? 2 : 3})), k(kind_of(x, "x")), B(size(x.size(0), "B")), L(one ? 1 : size(x.size(1), "L")),
          C(size(x.size(-1), "C")), K(0), w(nullptr), bias(nullptr) {
        const Tensor &t = ranked(ow, "weight", {2});
        K = size(t.size(1), "K");
        w = static_cast<const float *>(ptr(check(ow, "weight", {C, K}, at::kFloat, k)));
        bias = opt<const float>(ob, "bias", {C}, at::kFloat, k);
    }
    Shape state() const { return {B, K > 0 ? K - 1 : 0, C}; }
};

// x, weight, bias, state, act, lens, y, state_out
PyObject *conv_forward(PyObject *const *a) {
    const ConvIn in(a[0], a[1], a[2], false);
    const void *state = opt(a[3], "state", in.state(), in.k.dt, in.k);
    const int *lens = opt<const int>(a[5], "lens", {in.B}, at::kInt, in.k);
    const Tensor y = output(a[6], "y", in.x.sizes(), in.k.dt, in.k, false);
    const Tensor so = output(a[7], "state_out", in.state(), in.k.dt, in.k);
    const Operand ox(in.x, "x"), oy(y, "y");
    const int act = number(a[4]);
    call(in.k, [&](hipStream_t s) {
        return ttt_conv_forward(in.B, in.L, in.C, in.K, in.k.io, act, ox.p, ox.strides, in.w, in.bias, state, lens, oy.p,
                                oy.strides, ptr(so), s);
    });
    written(a[6], y);
    written(a[7], so);
    return pair(y, so);
}

// x, weight, state, bias, act, y
PyObject *conv_step(PyObject *const *a) {
    const ConvIn in(a[0], a[1], a[3], true);
    const Tensor &state = check(a[2], "state", in.state(), in.k.dt, in.k);
    const Tensor y = output(a[5], "y", in.x.sizes(), in.k.dt, in.k);
    const Operand ox(in.x, "x");
    const int act = number(a[4]);
    call(in.k, [&](hipStream_t s) {
        return ttt_conv_step(in.B, in.C, in.K, in.k.io, act, ox.p, ox.strides, in.w, in.bias, ptr(state), ptr(y), s);
    });
    written(state);
    written(a[5], y);
    return THPVariable_Wrap(y);
}

// x, weight, dy, bias, state, dstate_out, act, lens, workspace, grads
PyObject *conv_backward(PyObject *const *a) {
    const ConvIn in(a[0], a[1], a[3], false);
    const Tensor &dy = check(a[2], "dy", in.x.sizes(), in.k.dt, in.k, false);
    const void *state = opt(a[4], "state", in.state(), in.k.dt, in.k);
    const void *dso = opt(a[5], "dstate_out", in.state(), in.k.dt, in.k);
    const int *lens = opt<const int>(a[7], "lens", {in.B}, at::kInt, in.k);
    Grads g(a[9], in.k);
    const Tensor dx = g.get("dx", in.x.sizes(), in.k.dt, false), dw = g.get("dweight", {in.C, in.K}, at::kFloat);
    Tensor db, ds;
    if (a[3] != Py_None) db = g.get("dbias", {in.C}, at::kFloat);
    if (a[4] != Py_None) ds = g.get("dstate", in.state(), in.k.dt);
    g.whole();
    size_t need = 0;
    done(ttt_conv_backward_workspace(in.B, in.L, in.C, in.K, &need));
    const Workspace ws(a[8], need, in.k);
    const Operand ox(in.x, "x"), oy(dy, "dy"), od(dx, "dx");
    const int act = number(a[6]);
    call(in.k, [&](hipStream_t s) {
        return ttt_conv_backward(in.B, in.L, in.C, in.K, in.k.io, act, ox.p, ox.strides, in.w, in.bias, state, lens, oy.p,
                                 oy.strides, dso, od.p, od.strides, static_cast<float *>(ptr(dw)),
                                 db.defined() ? static_cast<float *>(ptr(db)) : nullptr, ds.defined() ? ptr(ds) : nullptr,
                                 ws.p, ws.bytes, s);
    });
    return g.take();
}

// --- state space scan ----------------------------------------------------------

// x, dt, A, B, C, D, dt_bias
struct ScanIn {
    const Tensor &x;
    Kind k;
    int B, L, H, P, G, N;
    const Tensor &dt, &Bm, &Cm;
    const float *A, *D, *dt_bias;
    Operand ox, odt, ob, oc;
    static Shape lead(const Tensor &x, std::initializer_list<int64_t> tail) {
        Shape s(x.sizes().begin(), x.sizes().end() - 2);
        s.insert(s.end(), tail);
        return s;
    }
    ScanIn(PyObject *const *a, PyObject *oD, PyObject *obias, bool one)
        : x(ranked(a[0], "x", {one ? 3 : 4})), k(kind_of(x, "x")), B(size(x.size(0), "B")), L(one ? 1 : size(x.size(1), "L")),
          H(size(x.size(-2), "H")), P(size(x.size(-1), "P")), G(size(ranked(a[3], "B", {x.dim()}).size(-2), "G")),
          N(size(tensor(a[3], "B").size(-1), "N")), dt(check(a[1], "dt", lead(x, {H}), k.dt, k, false)),
          Bm(check(a[3], "B", lead(x, {G, N}), k.dt, k, false)), Cm(check(a[4], "C", lead(x, {G, N}), k.dt, k, false)),
          A(static_cast<const float *>(ptr(check(a[2], "A", {H}, at::kFloat, k)))), D(opt<const float>(oD, "D", {H}, at::kFloat, k)),
          dt_bias(opt<const float>(obias, "dt_bias", {H}, at::kFloat, k)), ox(x, "x"), odt(dt, "dt", 0), ob(Bm, "B"), oc(Cm, "C") {}
    Shape state() const { return {B, H, N, P}; }
};

// x, dt, A, B, C, D, dt_bias, state, lens, y, state_out, workspace
PyObject *ssm_forward(PyObject *const *a) {
    const ScanIn in(a, a[5], a[6], false);
    const float *state = opt<const float>(a[7], "state", in.state(), at::kFloat, in.k);
    const int *lens = opt<const int>(a[8], "lens", {in.B}, at::kInt, in.k);
    const Tensor y = output(a[9], "y", in.x.sizes(), in.k.dt, in.k, false);
    const Tensor so = output(a[10], "state_out", in.state(), at::kFloat, in.k);
    size_t need = 0;
    done(ttt_ssm_forward_workspace(in.B, in.L, in.H, in.P, in.G, in.N, &need));
    const Workspace ws(a[11], need, in.k);
    const Operand oy(y, "y");
    call(in.k, [&](hipStream_t s) {
        return ttt_ssm_forward(in.B, in.L, in.H, in.P, in.G, in.N, in.k.io, in.ox.p, in.ox.strides, in.odt.p, in.odt.strides,
                               in.A, in.ob.p, in.ob.strides, in.oc.p, in.oc.strides, in.D, in.dt_bias, state, lens, oy.p,
                               oy.strides, static_cast<float *>(ptr(so)), ws.p, ws.bytes, s);
    });
    written(a[9], y);
    written(a[10], so);
    return pair(y, so);
}

// x, dt, A, B, C, state, D, dt_bias, y
PyObject *ssm_step(PyObject *const *a) {
    const ScanIn in(a, a[6], a[7], true);
    const Tensor &state = check(a[5], "state", in.state(), at::kFloat, in.k);
    const Tensor y = output(a[8], "y", in.x.sizes(), in.k.dt, in.k);
    call(in.k, [&](hipStream_t s) {
        return ttt_ssm_step(in.B, in.H, in.P, in.G, in.N, in.k.io, in.ox.p, in.ox.strides, in.odt.p, in.odt.strides, in.A,
                            in.ob.p, in.ob.strides, in.oc.p, in.oc.strides, in.D, in.dt_bias, static_cast<float *>(ptr(state)),
                            ptr(y), s);
    });
    written(state);
    written(a[8], y);
    return THPVariable_Wrap(y);
}

// x, dt, A, B, C, dy, D, dt_bias, state, dstate_out, lens, workspace, grads
PyObject *ssm_backward(PyObject *const *a) {
    const ScanIn in(a, a[6], a[7], false);
    const Tensor &dy = check(a[5], "dy", in.x.sizes(), in.k.dt, in.k, false);
    const float *state = opt<const float>(a[8], "state", in.state(), at::kFloat, in.k);
    const float *dso = opt<const float>(a[9], "dstate_out", in.state(), at::kFloat, in.k);
    const int *lens = opt<const int>(a[10], "lens", {in.B}, at::kInt, in.k);
    Grads g(a[12], in.k);
    const Tensor dx = g.get("dx", in.x.sizes(), in.k.dt, false), ddt = g.get("ddt", in.dt.sizes(), in.k.dt, false),
                 dA = g.get("dA", {in.H}, at::kFloat), dB = g.get("dB", in.Bm.sizes(), in.k.dt, false),
                 dC = g.get("dC", in.Cm.sizes(), in.k.dt, false);
    Tensor dD, db, ds;
    if (a[6] != Py_None) dD = g.get("dD", {in.H}, at::kFloat);
    if (a[7] != Py_None) db = g.get("ddt_bias", {in.H}, at::kFloat);
    if (a[8] != Py_None) ds = g.get("dstate", in.state(), at::kFloat);
    g.whole();
    auto f = [](const Tensor &t) { return t.defined() ? static_cast<float *>(ptr(t)) : nullptr; };
    size_t need = 0;
    done(ttt_ssm_backward_workspace(in.B, in.L, in.H, in.P, in.G, in.N, &need));
    const Workspace ws(a[11], need, in.k);
    const Operand oy(dy, "dy"), odx(dx, "dx"), oddt(ddt, "ddt", 0), odb(dB, "dB"), odc(dC, "dC");
    call(in.k, [&](hipStream_t s) {
        return ttt_ssm_backward(in.B, in.L, in.H, in.P, in.G, in.N, in.k.io, in.ox.p, in.ox.strides, in.odt.p, in.odt.strides,
                                in.A, in.ob.p, in.ob.strides, in.oc.p, in.oc.strides, in.D, in.dt_bias, state, lens, oy.p,
                                oy.strides, dso, odx.p, odx.strides, oddt.p, oddt.strides, f(dA), odb.p, odb.strides, odc.p,
                                odc.strides, f(dD), f(db), f(ds), ws.p, ws.bytes, s);
    });
    return g.take();
}

// --- block norm ------------------------------------------------------------------

// resid, y, post_gamma, pre_gamma, gate, scale, post_beta, pre_beta, layer, act, eps, lens
struct NormIn {
    const Tensor &y, &resid;
    Kind k;
    int B, L, D, rio, shape;
    const Tensor *gate;
    const float *pg, *qg, *sc, *pb, *qb;
    int layer, act;
    float eps;
    const int *lens;
    Operand orr, oy;
    std::optional<Operand> og;
    explicit NormIn(PyObject *const *a)
        : y(ranked(a[1], "y", {3})), resid(tensor(a[0], "resid")), k(kind_of(y, "y")), B(size(y.size(0), "B")),
          L(size(y.size(1), "L")), D(size(y.size(2), "D")), rio(io_of(resid, "resid")), shape(TTT_GATE_NONE), gate(nullptr),
          pg(opt<const float>(a[2], "post_gamma", {D}, at::kFloat, k)), qg(opt<const float>(a[3], "pre_gamma", {D}, at::kFloat, k)),
          sc(opt<const float>(a[5], "scale", {D}, at::kFloat, k)), pb(opt<const float>(a[6], "post_beta", {D}, at::kFloat, k)),
          qb(opt<const float>(a[7], "pre_beta", {D}, at::kFloat, k)), layer(number(a[8])), act(number(a[9])),
          eps(static_cast<float>(PyFloat_AsDouble(a[10]))), lens(opt<const int>(a[11], "lens", {B}, at::kInt, k)),
          orr(check(a[0], "resid", y.sizes(), resid.scalar_type(), k, false), "resid"), oy(y, "y") {
        if (PyErr_Occurred()) throw PyError{};
        if (a[4] == Py_None) return;
        gate = &tensor(a[4], "gate");
        if (gate->dim() < 1 || gate->dim() > 3)
            raise(PyExc_ValueError, "gate has " + std::to_string(gate->dim()) + " dimensions, expected [D], [B,D] or [B,L,D]");
        shape = static_cast<int>(gate->dim());  // TTT_GATE_CHANNEL, _SEQUENCE, _TOKEN
        if (shape == TTT_GATE_TOKEN)
            check(a[4], "gate", y.sizes(), k.dt, k, false);
        else
            check(a[4], "gate", shape == TTT_GATE_CHANNEL ? Shape{D} : Shape{B, D}, at::kFloat, k);
        og.emplace(*gate, "gate");
    }
    const void *gp() const { return og ? og->p : nullptr; }
    const int64_t *gs() const { return og && shape == TTT_GATE_TOKEN ? og->strides : nullptr; }
};

// the twelve of NormIn, resid_out, x
PyObject *block_norm(PyObject *const *a) {
    const NormIn in(a);
    const Tensor ro = output(a[12], "resid_out", in.y.sizes(), in.resid.scalar_type(), in.k);
    const Tensor x = output(a[13], "x", in.y.sizes(), in.k.dt, in.k);
    call(in.k, [&](hipStream_t s) {
        return ttt_block_norm(in.B, in.L, in.D, in.k.io, in.rio, in.layer, in.shape, in.act, in.eps, in.orr.p, in.orr.strides,
                              in.oy.p, in.oy.strides, in.gp(), in.gs(), in.pg, in.pb, in.qg, in.qb, in.sc, in.lens, ptr(ro),
                              ptr(x), s);
    });
    written(a[12], ro);
    written(a[13], x);
    return pair(ro, x);
}

// the twelve of NormIn, dresid_out, dx, workspace, grads
PyObject *block_norm_backward(PyObject *const *a) {
    const NormIn in(a);
    const Tensor &dro = check(a[12], "dresid_out", in.y.sizes(), in.resid.scalar_type(), in.k);
    const Tensor &dx = check(a[13], "dx", in.y.sizes(), in.k.dt, in.k);
    Grads g(a[15], in.k);
    const Tensor dr = g.get("dresid", in.y.sizes(), in.resid.scalar_type()), dy = g.get("dy", in.y.sizes(), in.k.dt);
    Tensor dg, dp[5];
    if (in.gate) dg = g.get("dgate", in.gate->sizes(), in.gate->scalar_type());
    const char *names[5] = {"dpost_gamma", "dpre_gamma", "dpost_beta", "dpre_beta", "dscale"};
    const int from[5] = {2, 3, 6, 7, 5};
    float *q[5];
    for (int i = 0; i < 5; ++i) {
        if (a[from[i]] != Py_None) dp[i] = g.get(names[i], {in.D}, at::kFloat);
        q[i] = dp[i].defined() ? static_cast<float *>(ptr(dp[i])) : nullptr;
    }
    g.whole();
    size_t need = 0;
    done(ttt_block_norm_backward_workspace(in.B, in.L, in.D, in.shape, &need));
    const Workspace ws(a[14], need, in.k);
    call(in.k, [&](hipStream_t s) {
        return ttt_block_norm_backward(in.B, in.L, in.D, in.k.io, in.rio, in.layer, in.shape, in.act, in.eps, in.orr.p,
                                       in.orr.strides, in.oy.p, in.oy.strides, in.gp(), in.gs(), in.pg, in.pb, in.qg, in.qb,
                                       in.sc, in.lens, ptr(dro), ptr(dx), ptr(dr), ptr(dy), dg.defined() ? ptr(dg) : nullptr,
                                       q[0], q[2], q[1], q[3], q[4], ws.p, ws.bytes, s);
    });
    return g.take();
}

// --- gated linear recurrence -----------------------------------------------------

// x, r, rate, i
struct LruIn {
    const Tensor &x;
    Kind k;
    int B, L, D;
    const Tensor &r;
    const Tensor *i;
    const float *rate;
    Operand ox, orr;
    std::optional<Operand> oi;
    LruIn(PyObject *px, PyObject *pr, PyObject *prate, PyObject *pi, bool one)
        : x(ranked(px, "x", {one ? 2 : 3})), k(kind_of(x, "x")), B(size(x.size(0), "B")), L(one ? 1 : size(x.size(1), "L")),
          D(size(x.size(-1), "D")), r(check(pr, "r", x.sizes(), k.dt, k, false)), i(nullptr),
          rate(opt<const float>(prate, "rate", {D}, at::kFloat, k)), ox(x, "x"), orr(r, "r") {
        if (pi == Py_None) return;
        i = &check(pi, "i", x.sizes(), k.dt, k, false);
        oi.emplace(*i, "i");
    }
    const void *ip() const { return oi ? oi->p : nullptr; }
    const int64_t *is() const { return oi ? oi->strides : nullptr; }
    Shape state() const { return {B, D}; }
};

// x, r, rate, i, state, lens, y, state_out, workspace
PyObject *lru_forward(PyObject *const *a) {
    const LruIn in(a[0], a[1], a[2], a[3], false);
    const float *state = opt<const float>(a[4], "state", in.state(), at::kFloat, in.k);
    const int *lens = opt<const int>(a[5], "lens", {in.B}, at::kInt, in.k);
    const Tensor y = output(a[6], "y", in.x.sizes(), in.k.dt, in.k, false);
    const Tensor so = output(a[7], "state_out", in.state(), at::kFloat, in.k);
    size_t need = 0;
    done(ttt_lru_forward_workspace(in.B, in.L, in.D, &need));
    const Workspace ws(a[8], need, in.k);
    const Operand oy(y, "y");
    call(in.k, [&](hipStream_t s) {
        return ttt_lru_forward(in.B, in.L, in.D, in.k.io, in.ox.p, in.ox.strides, in.orr.p, in.orr.strides, in.ip(), in.is(),
                               in.rate, state, lens, oy.p, oy.strides, static_cast<float *>(ptr(so)), ws.p, ws.bytes, s);
    });
    written(a[6], y);
    written(a[7], so);
    return pair(y, so);
}

// x, r, state, rate, i, y
PyObject *lru_step(PyObject *const *a) {
    const LruIn in(a[0], a[1], a[3], a[4], true);
    const Tensor &state = check(a[2], "state", in.state(), at::kFloat, in.k);
    const Tensor y = output(a[5], "y", in.x.sizes(), in.k.dt, in.k);
    call(in.k, [&](hipStream_t s) {
        return ttt_lru_step(in.B, in.D, in.k.io, in.ox.p, in.ox.strides, in.orr.p, in.orr.strides, in.ip(), in.is(), in.rate,
                            static_cast<float *>(ptr(state)), ptr(y), s);
    });
    written(state);
    written(a[5], y);
    return THPVariable_Wrap(y);
}

// x, r, dy, rate, i, state, dstate_out, lens, workspace, grads
PyObject *lru_backward(PyObject *const *a) {
    const LruIn in(a[0], a[1], a[3], a[4], false);
    const Tensor &dy = check(a[2], "dy", in.x.sizes(), in.k.dt, in.k, false);
    const float *state = opt<const float>(a[5], "state", in.state(), at::kFloat, in.k);
    const float *dso = opt<const float>(a[6], "dstate_out", in.state(), at::kFloat, in.k);
    const int *lens = opt<const int>(a[7], "lens", {in.B}, at::kInt, in.k);
    Grads g(a[9], in.k);
    const Tensor dx = g.get("dx", in.x.sizes(), in.k.dt, false), dr = g.get("dr", in.x.sizes(), in.k.dt, false);
    Tensor di, dq, ds;
    if (in.i) di = g.get("di", in.x.sizes(), in.k.dt, false);
    if (a[3] != Py_None) dq = g.get("drate", {in.D}, at::kFloat);
    if (a[5] != Py_None) ds = g.get("dstate", in.state(), at::kFloat);
    g.whole();
    auto f = [](const Tensor &t) { return t.defined() ? static_cast<float *>(ptr(t)) : nullptr; };
    size_t need = 0;
    done(ttt_lru_backward_workspace(in.B, in.L, in.D, &need));
    const Workspace ws(a[8], need, in.k);
    const Operand oy(dy, "dy"), odx(dx, "dx"), odr(dr, "dr");
    std::optional<Operand> odi;
    if (in.i) odi.emplace(di, "di");
    call(in.k, [&](hipStream_t s) {
        return ttt_lru_backward(in.B, in.L, in.D, in.k.io, in.ox.p, in.ox.strides, in.orr.p, in.orr.strides, in.ip(), in.is(),
                                in.rate, state, lens, oy.p, oy.strides, dso, odx.p, odx.strides, odr.p, odr.strides,
                                odi ? odi->p : nullptr, odi ? odi->strides : nullptr, f(dq), f(ds), ws.p, ws.bytes, s);
    });
    return g.take();
}

// --- products in 8-bit integers ----------------------------------------------------

// rows of the innermost dimension: all others as one, by one stride
struct RowsOf {
    const Tensor &t;
    int M, K;
    int64_t stride;
    Shape lead;
    RowsOf(const Tensor &x, const char *name) : t(x), M(0), K(0), stride(0) {
        if (t.dim() < 1) raise(PyExc_ValueError, std::string(name) + " has no dimension");
        lead.assign(t.sizes().begin(), t.sizes().end() - 1);
        K = size(t.size(-1), "K");
        if (K > 1 && t.stride(-1) != 1)
            raise(PyExc_ValueError, std::string("the innermost dimension of ") + name + " must be contiguous");
        int64_t n = 1;
        stride = K;
        for (int64_t i = t.dim() - 2; i >= 0; --i) {
            if (t.size(i) == 1) continue;
            if (n == 1)
                stride = t.stride(i);
            else if (n && t.stride(i) != n * stride)
                raise(PyExc_ValueError, "the rows of " + std::string(name) + " are not one stride apart");
            n *= t.size(i);
        }
        M = size(n, "M");
    }
    RowsOf(const RowsOf &) = delete;
    Shape with(int64_t inner) const {
        Shape s = lead;
        s.push_back(inner);
        return s;
    }
};

Kind on_device(const Tensor &t, const char *name, at::ScalarType dt) {
    if (t.scalar_type() != dt)
        raise(PyExc_TypeError, std::string(name) + " has dtype " + text(t.scalar_type()) + ", expected " + text(dt));
    if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a device tensor (got " + t.device().str() + ")");
    return {static_cast<int>(t.get_device()), dt, 0};
}

// x, q, scale
PyObject *i8_quantize(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x");
    const Kind k = kind_of(x, "x");
    const RowsOf r(x, "x");
    const Tensor q = output(a[1], "q", x.sizes(), at::kChar, k, false), scale = output(a[2], "scale", r.lead, at::kFloat, k);
    const RowsOf rq(q, "q");
    call(k, [&](hipStream_t s) {
        return ttt_i8_quantize(r.M, r.K, k.io, ptr(x), &r.stride, static_cast<int8_t *>(ptr(q)), &rq.stride,
                               static_cast<float *>(ptr(scale)), s);
    });
    written(a[1], q);
    written(a[2], scale);
    return pair(q, scale);
}

// w, w_scale, bias
struct I8Weight {
    const RowsOf w;
    const float *scale, *bias;
    I8Weight(PyObject *pw, PyObject *ps, PyObject *pb, int64_t K, const Kind &k)
        : w(check(pw, "w", {ranked(pw, "w", {2}).size(0), K}, at::kChar, k, false), "w"),
          scale(static_cast<const float *>(ptr(check(ps, "w_scale", {w.M}, at::kFloat, k)))),
          bias(opt<const float>(pb, "bias", {w.M}, at::kFloat, k)) {}
};

// x, x_scale, w, w_scale, bias, bf16, y, workspace
PyObject *i8_project(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x");
    const Kind k = on_device(x, "x", at::kChar);
    const RowsOf r(x, "x");
    const float *xs = static_cast<const float *>(ptr(check(a[1], "x_scale", r.lead, at::kFloat, k)));
    const I8Weight w(a[2], a[3], a[4], r.K, k);
    const int io = number(a[5]);
    const Tensor y = output(a[6], "y", r.with(w.w.M), io == TTT_BF16 ? at::kBFloat16 : at::kFloat, k, false);
    const RowsOf ry(y, "y");
    const int8_t *px = static_cast<const int8_t *>(ptr(x)), *pw = static_cast<const int8_t *>(ptr(w.w.t));
    size_t need = 0;
    done(ttt_i8_project_workspace(r.M, r.K, w.w.M, px, &r.stride, pw, &w.w.stride, &need));
    const Workspace ws(a[7], need, k);
    call(k, [&](hipStream_t s) {
        return ttt_i8_project(r.M, r.K, w.w.M, io, px, &r.stride, xs, pw, &w.w.stride, w.scale, w.bias, ptr(y), &ry.stride,
                              ws.p, ws.bytes, s);
    });
    written(a[6], y);
    return THPVariable_Wrap(y);
}

// x, w, w_scale, bias, y, workspace
PyObject *i8_linear(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x");
    const Kind k = kind_of(x, "x");
    const RowsOf r(x, "x");
    const I8Weight w(a[1], a[2], a[3], r.K, k);
    const Tensor y = output(a[4], "y", r.with(w.w.M), k.dt, k, false);
    const RowsOf ry(y, "y");
    const int8_t *pw = static_cast<const int8_t *>(ptr(w.w.t));
    size_t need = 0;
    done(ttt_i8_linear_workspace(r.M, r.K, w.w.M, pw, &w.w.stride, &need));
    const Workspace ws(a[5], need, k);
    call(k, [&](hipStream_t s) {
        return ttt_i8_linear(r.M, r.K, w.w.M, k.io, ptr(x), &r.stride, pw, &w.w.stride,
                             w.scale, w.bias, ptr(y), &ry.stride, ws.p, ws.bytes, s);
    });
    written(a[4], y);
    return THPVariable_Wrap(y);
}

// X, theta, theta_scale, H, out (None or a tuple of three), workspace
PyObject *qkv_project_i8(PyObject *const *a) {
    const Tensor &x = ranked(a[0], "X", {3});
    const Kind k = on_device(x, "X", at::kBFloat16);
    const int B = size(x.size(0), "B"), L = size(x.size(1), "L"), dm = size(x.size(2), "d_model");
    const long heads = PyLong_AsLong(a[3]);
    if (heads == -1 && PyErr_Occurred()) throw PyError{};
    if (heads < 0) raise(PyExc_ValueError, "H = " + std::to_string(heads) + " is negative");
    const int H = size(heads, "H");
    const int64_t hd = static_cast<int64_t>(H) * 64;
    check(a[0], "X", x.sizes(), at::kBFloat16, k);
    const Tensor &th = check(a[1], "theta", {3, hd, dm}, at::kChar, k), &ts = check(a[2], "theta_scale", {3, hd}, at::kFloat, k);
    if (a[4] != Py_None && (!PyTuple_Check(a[4]) || PyTuple_GET_SIZE(a[4]) != 3))
        raise(PyExc_ValueError, "out must be a tuple of three tensors");
    const char *names[3] = {"XQ", "XK", "XV"};
    Tensor out[3];
    for (int i = 0; i < 3; ++i)
        out[i] = output(a[4] == Py_None ? Py_None : PyTuple_GET_ITEM(a[4], i), names[i], {B, H, L, 64}, at::kBFloat16, k);
    size_t need = 0;
    const int8_t *pt = static_cast<const int8_t *>(ptr(th));
    done(ttt_i8_linear_workspace(size(static_cast<int64_t>(B) * L, "B*L"), dm, size(3 * hd, "3*H*64"), pt, nullptr, &need));
    const Workspace ws(a[5], need, k);
    call(k, [&](hipStream_t s) {
        return ttt_qkv_project_i8(B, L, dm, H, 64, ptr(x), pt,
                                  static_cast<const float *>(ptr(ts)), ptr(out[0]), ptr(out[1]), ptr(out[2]), ws.p, ws.bytes, s);
    });
    PyObject *r = PyTuple_New(3);
    for (int i = 0; r && i < 3; ++i) {
        if (a[4] != Py_None) written(out[i]);
        PyObject *o = THPVariable_Wrap(out[i]);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i, o);
    }
    return r;
}

// the class that errors of the C ABI are raised as
PyObject *init(PyObject *const *a) {
    Py_XDECREF(ttt_error);
    ttt_error = a[0];
    Py_INCREF(ttt_error);
    Py_RETURN_NONE;
}

#define METHOD(name, n) \
    { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&method<name, n>)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {METHOD(init, 1), METHOD(conv_forward, 8), METHOD(conv_step, 6), METHOD(conv_backward, 10),
                         METHOD(ssm_forward, 12), METHOD(ssm_step, 9), METHOD(ssm_backward, 13), METHOD(block_norm, 14),
                         METHOD(block_norm_backward, 16), METHOD(lru_forward, 9), METHOD(lru_step, 6),
                         METHOD(lru_backward, 10), METHOD(i8_quantize, 3), METHOD(i8_project, 8), METHOD(i8_linear, 6),
                         METHOD(qkv_project_i8, 6), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block(void) { return PyModule_Create(&module); }
