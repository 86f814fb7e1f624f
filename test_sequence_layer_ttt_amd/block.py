"""Python binding of the operators around the layer: the short causal
convolution, the selective state space scan and the block norm, under the C
ABI's names (ttt.py offers them too).

Argument marshalling only, as in ttt.py, with two differences that the ABI
makes possible: operands may be strided views (innermost dimension contiguous)
and the call runs on the operands' device, whichever device is current. A
`stream` that is given must be one of that device.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import _lib

_IO = {torch.float32: _lib.TTT_F32, torch.bfloat16: _lib.TTT_BF16}
_ACT = {"none": _lib.TTT_ACT_NONE, "sigmoid": _lib.TTT_ACT_SIGMOID, "silu": _lib.TTT_ACT_SILU,
        "tanh": _lib.TTT_ACT_TANH}
_S1, _S2, _S3 = (ctypes.c_int64 * n for n in (1, 2, 3))


def _io(t, name: str):
    """(storage type, device number) of an operand that sets both."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    io = _IO.get(t.dtype)
    if io is None:
        raise TypeError(f"{name} dtype {t.dtype} not supported")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    return io, t.get_device()


def _check(t, name: str, shape, dtype, index: int, contiguous: bool = True) -> None:
    """`index`: the device's number (a tensor's own is quicker to ask than its device)."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
            and (not contiguous or t.is_contiguous())):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    raise ValueError(f"{name} must be contiguous")


def _rows(t, name: str, kind, skip: int = 1):
    """The strides of all but the innermost `skip` dimensions as a host array;
    None where the tensor is contiguous."""
    if t.is_contiguous():
        return None
    if skip and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"the innermost dimension of {name} must be contiguous")
    s = t.stride()
    return kind(*(s[:-1] if skip else s))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr() or None


def _call(fn, index: int, stream, *args) -> None:
    """The entry point on device `index` and its current stream, or on `stream`."""
    if stream is None:
        raw = _raw_stream(index)
    else:
        if isinstance(stream, torch.cuda.Stream) and stream.device.index != index:
            raise ValueError(f"stream is on {stream.device}, the operands on cuda:{index}")
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if index == _current_device():
        code = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            code = fn(*args, raw)
    if code:
        _lib.check(code)


# The handle of a device's current stream and the current device's number,
# without the objects that torch.cuda's functions make of them (2.5 us a call);
# a tensor on the device exists, so it is initialised.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _lens(lens, B, index: int):
    if lens is None:
        return None
    _check(lens, "lens", (B,), torch.int32, index)
    return _ptr(lens)


def _workspace(workspace, need: int, index: int):
    if workspace is None:
        if not need:
            return None, 0
        workspace = torch.empty(need, device=_device(index), dtype=torch.uint8)
        return workspace, need
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the operands' device")
    return workspace, workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=4096)
def _need(name: str, *args) -> int:
    """A workspace query's answer, which goes by the sizes alone."""
    n = ctypes.c_size_t(0)
    _lib.check(getattr(_lib.load(), name)(*args, ctypes.byref(n)))
    return n.value


def _grads(grads, index: int, shapes: dict) -> dict:
    """The outputs of a backward: `grads` as given, or new contiguous ones."""
    if grads is None:
        return {k: _new(s, t, index) for k, (s, t) in shapes.items()}
    if set(grads) != set(shapes):
        raise ValueError(f"grads has {sorted(grads)}, expected {sorted(shapes)}")
    for k, (s, t) in shapes.items():
        _check(grads[k], k, s, t, index, contiguous=False)
    return grads


@functools.lru_cache(maxsize=None)
def _device(index: int) -> torch.device:
    return torch.device("cuda", index)


def _new(shape, dtype, index: int):
    return torch.empty(shape, device=_device(index), dtype=dtype)


def _plain(g, name):
    t = g.get(name)
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _ptr(t)


# --- short causal convolution ------------------------------------------------


def _conv_act(activation: str) -> int:
    if activation not in ("none", "silu"):
        raise ValueError(f"activation {activation!r} is not 'none' or 'silu'")
    return _ACT[activation]


def ttt_conv_forward(x, weight, bias=None, state=None, activation: str = "silu", lens=None, y=None,
                     state_out=None, stream=None):
    """Causal convolution over the last K tokens of each channel, K in 2..4:
    y_t = act(bias + sum_k weight[:, k] x_{t-K+1+k}). x, y [B,L,C] (fp32 or
    bf16, views with a contiguous last dimension allowed), weight [C,K] and
    bias [C] fp32, state [B,K-1,C] the tokens before the first (zeros if
    None), activation "silu" or "none", lens [B] int32 optional lengths.
    Returns (y, state_out); state_out may be `state` itself."""
    io, dev = _io(x, "x")
    B, L, C = x.shape
    K = weight.shape[-1]
    _check(weight, "weight", (C, K), torch.float32, dev)
    if bias is not None:
        _check(bias, "bias", (C,), torch.float32, dev)
    if state is not None:
        _check(state, "state", (B, K - 1, C), x.dtype, dev)
    if y is None:
        y = _new((B, L, C), x.dtype, dev)
    if state_out is None:
        state_out = _new((B, K - 1, C), x.dtype, dev)
    _check(y, "y", (B, L, C), x.dtype, dev, contiguous=False)
    _check(state_out, "state_out", (B, K - 1, C), x.dtype, dev)
    _call(_lib.load().ttt_conv_forward, dev, stream, B, L, C, K, io, _conv_act(activation), _ptr(x),
          _rows(x, "x", _S2), _ptr(weight), _ptr(bias), _ptr(state), _lens(lens, B, dev), _ptr(y),
          _rows(y, "y", _S2), _ptr(state_out))
    return y, state_out


def ttt_conv_step(x, weight, state, bias=None, activation: str = "silu", y=None, stream=None):
    """One token of ttt_conv_forward for each sequence: x [B,C] (a view with a
    contiguous last dimension allowed), state [B,K-1,C] updated in place.
    Returns y [B,C]."""
    io, dev = _io(x, "x")
    B, C = x.shape
    K = weight.shape[-1]
    _check(weight, "weight", (C, K), torch.float32, dev)
    if bias is not None:
        _check(bias, "bias", (C,), torch.float32, dev)
    _check(state, "state", (B, K - 1, C), x.dtype, dev)
    if y is None:
        y = _new((B, C), x.dtype, dev)
    _check(y, "y", (B, C), x.dtype, dev)
    _call(_lib.load().ttt_conv_step, dev, stream, B, C, K, io, _conv_act(activation), _ptr(x),
          _rows(x, "x", _S1), _ptr(weight), _ptr(bias), _ptr(state), _ptr(y))
    return y


def ttt_conv_backward_workspace(B: int, L: int, C: int, K: int) -> int:
    """Bytes of device workspace ttt_conv_backward needs."""
    return _need("ttt_conv_backward_workspace", B, L, C, K)


def ttt_conv_backward(x, weight, dy, bias=None, state=None, dstate_out=None, activation: str = "silu",
                      lens=None, workspace=None, grads=None, stream=None) -> dict:
    """Gradients of <dy, y> + <dstate_out, state_out> through ttt_conv_forward:
    dx [B,L,C] in x's type, dweight [C,K] fp32, with a bias dbias [C] fp32 and
    with a state dstate [B,K-1,C] in x's type. `grads` may hold the outputs
    (a dict like the one returned; dx may be strided)."""
    io, dev = _io(x, "x")
    B, L, C = x.shape
    K = weight.shape[-1]
    _check(weight, "weight", (C, K), torch.float32, dev)
    _check(dy, "dy", (B, L, C), x.dtype, dev, contiguous=False)
    shapes = {"dx": ((B, L, C), x.dtype), "dweight": ((C, K), torch.float32)}
    if bias is not None:
        _check(bias, "bias", (C,), torch.float32, dev)
        shapes["dbias"] = ((C,), torch.float32)
    if state is not None:
        _check(state, "state", (B, K - 1, C), x.dtype, dev)
        shapes["dstate"] = ((B, K - 1, C), x.dtype)
    if dstate_out is not None:
        _check(dstate_out, "dstate_out", (B, K - 1, C), x.dtype, dev)
    g = _grads(grads, dev, shapes)
    workspace, nbytes = _workspace(workspace, ttt_conv_backward_workspace(B, L, C, K), dev)
    _call(_lib.load().ttt_conv_backward, dev, stream, B, L, C, K, io, _conv_act(activation), _ptr(x),
          _rows(x, "x", _S2), _ptr(weight), _ptr(bias), _ptr(state), _lens(lens, B, dev), _ptr(dy),
          _rows(dy, "dy", _S2), _ptr(dstate_out), _ptr(g["dx"]), _rows(g["dx"], "dx", _S2),
          _plain(g, "dweight"), _plain(g, "dbias"), _plain(g, "dstate"), _ptr(workspace), nbytes)
    return g


# --- selective state space scan -------------------------------------------------


def _ssm_args(x, dt, A, B, C, D, dt_bias):
    """Checks and the operands' part of the argument list; B and C as given."""
    io, dev = _io(x, "x")
    lead, (H, P) = x.shape[:-2], x.shape[-2:]
    G, N = B.shape[-2:]
    kind = _S2 if x.dim() == 3 else _S3
    _check(dt, "dt", lead + (H,), x.dtype, dev, contiguous=False)
    _check(B, "B", lead + (G, N), x.dtype, dev, contiguous=False)
    _check(C, "C", lead + (G, N), x.dtype, dev, contiguous=False)
    _check(A, "A", (H,), torch.float32, dev)
    if D is not None:
        _check(D, "D", (H,), torch.float32, dev)
    if dt_bias is not None:
        _check(dt_bias, "dt_bias", (H,), torch.float32, dev)
    return dev, (*lead, H, P, G, N), (io, _ptr(x), _rows(x, "x", kind), _ptr(dt), _rows(dt, "dt", kind, 0),
                                      _ptr(A), _ptr(B), _rows(B, "B", kind), _ptr(C), _rows(C, "C", kind),
                                      _ptr(D), _ptr(dt_bias))


def ttt_ssm_forward_workspace(B: int, L: int, H: int, P: int, G: int, N: int) -> int:
    """Bytes of device workspace ttt_ssm_forward needs."""
    return _need("ttt_ssm_forward_workspace", B, L, H, P, G, N)


def ttt_ssm_forward(x, dt, A, B, C, D=None, dt_bias=None, state=None, lens=None, y=None, state_out=None,
                    workspace=None, stream=None):
    """Selective state space scan over [B,L,H,P] features: with d_t =
    softplus(dt_t + dt_bias), state <- exp(d_t A) state + B_t (d_t x_t)^T and
    y_t = C_t state + D x_t, a state [N,P] for each head. x, y [B,L,H,P], dt
    [B,L,H], B, C [B,L,G,N] in fp32 or bf16 (views allowed, the features
    contiguous; [B,H,L,d] features go in as x.transpose(1, 2)); A, D, dt_bias
    [H] fp32; state, state_out [B,H,N,P] fp32; lens [B] int32 optional lengths.
    Returns (y, state_out); state_out may be `state` itself."""
    dev, (Bn, L, H, P, G, N), args = _ssm_args(x, dt, A, B, C, D, dt_bias)
    if state is not None:
        _check(state, "state", (Bn, H, N, P), torch.float32, dev)
    if y is None:
        y = _new((Bn, L, H, P), x.dtype, dev)
    if state_out is None:
        state_out = _new((Bn, H, N, P), torch.float32, dev)
    _check(y, "y", (Bn, L, H, P), x.dtype, dev, contiguous=False)
    _check(state_out, "state_out", (Bn, H, N, P), torch.float32, dev)
    workspace, nbytes = _workspace(workspace, ttt_ssm_forward_workspace(Bn, L, H, P, G, N), dev)
    _call(_lib.load().ttt_ssm_forward, dev, stream, Bn, L, H, P, G, N, *args, _ptr(state),
          _lens(lens, Bn, dev), _ptr(y), _rows(y, "y", _S3), _ptr(state_out), _ptr(workspace), nbytes)
    return y, state_out


def ttt_ssm_step(x, dt, A, B, C, state, D=None, dt_bias=None, y=None, stream=None):
    """One token of ttt_ssm_forward for each sequence: x [B,H,P], dt [B,H], B,
    C [B,G,N] (views allowed), state [B,H,N,P] fp32 updated in place. Returns
    y [B,H,P]."""
    dev, (Bn, H, P, G, N), args = _ssm_args(x, dt, A, B, C, D, dt_bias)
    _check(state, "state", (Bn, H, N, P), torch.float32, dev)
    if y is None:
        y = _new((Bn, H, P), x.dtype, dev)
    _check(y, "y", (Bn, H, P), x.dtype, dev)
    _call(_lib.load().ttt_ssm_step, dev, stream, Bn, H, P, G, N, *args, _ptr(state), _ptr(y))
    return y


def ttt_ssm_backward_workspace(B: int, L: int, H: int, P: int, G: int, N: int) -> int:
    """Bytes of device workspace ttt_ssm_backward needs."""
    return _need("ttt_ssm_backward_workspace", B, L, H, P, G, N)


def ttt_ssm_backward(x, dt, A, B, C, dy, D=None, dt_bias=None, state=None, dstate_out=None, lens=None,
                     workspace=None, grads=None, stream=None) -> dict:
    """Gradients of <dy, y> + <dstate_out, state_out> through ttt_ssm_forward:
    dx, ddt, dB, dC shaped as their operands in x's type, dA [H] fp32 and, for
    those of D, dt_bias and state that are given, dD, ddt_bias [H] and dstate
    [B,H,N,P] fp32. `grads` may hold the outputs (a dict like the one
    returned; dx, ddt, dB, dC may be strided, slices of one buffer too)."""
    dev, (Bn, L, H, P, G, N), args = _ssm_args(x, dt, A, B, C, D, dt_bias)
    _check(dy, "dy", (Bn, L, H, P), x.dtype, dev, contiguous=False)
    shapes = {"dx": ((Bn, L, H, P), x.dtype), "ddt": ((Bn, L, H), x.dtype), "dA": ((H,), torch.float32),
              "dB": ((Bn, L, G, N), x.dtype), "dC": ((Bn, L, G, N), x.dtype)}
    if D is not None:
        shapes["dD"] = ((H,), torch.float32)
    if dt_bias is not None:
        shapes["ddt_bias"] = ((H,), torch.float32)
    if state is not None:
        _check(state, "state", (Bn, H, N, P), torch.float32, dev)
        shapes["dstate"] = ((Bn, H, N, P), torch.float32)
    if dstate_out is not None:
        _check(dstate_out, "dstate_out", (Bn, H, N, P), torch.float32, dev)
    g = _grads(grads, dev, shapes)
    workspace, nbytes = _workspace(workspace, ttt_ssm_backward_workspace(Bn, L, H, P, G, N), dev)
    _call(_lib.load().ttt_ssm_backward, dev, stream, Bn, L, H, P, G, N, *args, _ptr(state),
          _lens(lens, Bn, dev), _ptr(dy), _rows(dy, "dy", _S3), _ptr(dstate_out),
          _ptr(g["dx"]), _rows(g["dx"], "dx", _S3), _ptr(g["ddt"]), _rows(g["ddt"], "ddt", _S3, 0),
          _plain(g, "dA"), _ptr(g["dB"]), _rows(g["dB"], "dB", _S3), _ptr(g["dC"]),
          _rows(g["dC"], "dC", _S3), _plain(g, "dD"), _plain(g, "ddt_bias"), _plain(g, "dstate"),
          _ptr(workspace), nbytes)
    return g


# --- norms, gate and residual between two blocks -------------------------------


def _norm_args(resid, y, post_gamma, pre_gamma, gate, scale, post_beta, pre_beta, norm, gate_act, eps,
               lens):
    io, dev = _io(y, "y")
    B, L, D = y.shape
    rio, _ = _io(resid, "resid")
    _check(resid, "resid", (B, L, D), resid.dtype, dev, contiguous=False)
    if norm not in ("rms", "layer"):
        raise ValueError(f"norm {norm!r} is not 'rms' or 'layer'")
    if gate_act not in _ACT:
        raise ValueError(f"gate_act {gate_act!r} is not one of {sorted(_ACT)}")
    for t, n in ((post_gamma, "post_gamma"), (pre_gamma, "pre_gamma"), (post_beta, "post_beta"),
                 (pre_beta, "pre_beta"), (scale, "scale")):
        if t is not None:
            _check(t, n, (D,), torch.float32, dev)
    shape, gs = _lib.TTT_GATE_NONE, None
    if gate is not None:
        shape = {1: _lib.TTT_GATE_CHANNEL, 2: _lib.TTT_GATE_SEQUENCE, 3: _lib.TTT_GATE_TOKEN}.get(gate.dim())
        if shape is None:
            raise ValueError(f"gate has {gate.dim()} dimensions, expected [D], [B,D] or [B,L,D]")
        if shape == _lib.TTT_GATE_TOKEN:
            _check(gate, "gate", (B, L, D), y.dtype, dev, contiguous=False)
            gs = _rows(gate, "gate", _S2)
        else:
            _check(gate, "gate", (D,) if gate.dim() == 1 else (B, D), torch.float32, dev)
    return dev, shape, (B, L, D, io, rio, int(norm == "layer"), shape, _ACT[gate_act], eps, _ptr(resid),
                        _rows(resid, "resid", _S2), _ptr(y), _rows(y, "y", _S2), _ptr(gate), gs,
                        _ptr(post_gamma), _ptr(post_beta), _ptr(pre_gamma), _ptr(pre_beta), _ptr(scale),
                        _lens(lens, B, dev))


def ttt_block_norm(resid, y, post_gamma=None, pre_gamma=None, gate=None, scale=None, post_beta=None,
                   pre_beta=None, norm: str = "rms", gate_act: str = "none", eps: float = 1e-6, lens=None,
                   resid_out=None, x=None, stream=None):
    """Between two blocks of a stack: resid_out = scale resid + act(gate)
    (Norm(y) post_gamma + post_beta) and x = Norm(resid_out) pre_gamma +
    pre_beta, row by row. resid, y [B,L,D] (views with a contiguous last
    dimension allowed; resid fp32 or y's type); gate [D] or [B,D] fp32, or
    [B,L,D] in y's type; scale, gammas and betas [D] fp32; norm "rms" or
    "layer"; gate_act "none", "sigmoid", "silu" or "tanh".
    Returns (resid_out, x)."""
    dev, _, args = _norm_args(resid, y, post_gamma, pre_gamma, gate, scale, post_beta, pre_beta, norm,
                              gate_act, eps, lens)
    if resid_out is None:
        resid_out = _new(resid.shape, resid.dtype, dev)
    if x is None:
        x = _new(y.shape, y.dtype, dev)
    _check(resid_out, "resid_out", resid.shape, resid.dtype, dev)
    _check(x, "x", y.shape, y.dtype, dev)
    _call(_lib.load().ttt_block_norm, dev, stream, *args, _ptr(resid_out), _ptr(x))
    return resid_out, x


def ttt_block_norm_backward_workspace(B: int, L: int, D: int, gate_dims: int = 0) -> int:
    """Bytes of device workspace ttt_block_norm_backward needs (gate_dims: the
    gate's number of dimensions, 0 without a gate)."""
    return _need("ttt_block_norm_backward_workspace", B, L, D, gate_dims)


def ttt_block_norm_backward(resid, y, post_gamma, pre_gamma, dresid_out, dx, gate=None, scale=None,
                            post_beta=None, pre_beta=None, norm: str = "rms", gate_act: str = "none",
                            eps: float = 1e-6, lens=None, workspace=None, grads=None, stream=None) -> dict:
    """Gradients of <dresid_out, resid_out> + <dx, x> through ttt_block_norm,
    from its inputs. dresid_out and dresid in resid's type, dx and dy in y's,
    [B,L,D] contiguous; dgate shaped and typed as gate; dscale, dpost_gamma,
    dpre_gamma, dpost_beta, dpre_beta [D] fp32, of those parameters that are
    given. Returns them in a dict; `grads` may hold the outputs."""
    dev, shape, args = _norm_args(resid, y, post_gamma, pre_gamma, gate, scale, post_beta, pre_beta, norm,
                                  gate_act, eps, lens)
    B, L, D = y.shape
    _check(dresid_out, "dresid_out", resid.shape, resid.dtype, dev)
    _check(dx, "dx", y.shape, y.dtype, dev)
    shapes = {"dresid": (resid.shape, resid.dtype), "dy": (y.shape, y.dtype)}
    if gate is not None:
        shapes["dgate"] = (gate.shape, gate.dtype)
    for t, n in ((post_gamma, "dpost_gamma"), (pre_gamma, "dpre_gamma"), (post_beta, "dpost_beta"),
                 (pre_beta, "dpre_beta"), (scale, "dscale")):
        if t is not None:
            shapes[n] = ((D,), torch.float32)
    g = _grads(grads, dev, shapes)
    workspace, nbytes = _workspace(workspace, ttt_block_norm_backward_workspace(B, L, D, shape), dev)
    _call(_lib.load().ttt_block_norm_backward, dev, stream, *args, _ptr(dresid_out), _ptr(dx),
          _plain(g, "dresid"), _plain(g, "dy"), _plain(g, "dgate"), _plain(g, "dpost_gamma"),
          _plain(g, "dpost_beta"), _plain(g, "dpre_gamma"), _plain(g, "dpre_beta"), _plain(g, "dscale"),
          _ptr(workspace), nbytes)
    return g
