"""Python binding of the operators around the layer: the short causal
convolution, the selective state space scan, the gated linear recurrence, the
block norm and the 8-bit integer products, under the C ABI's names (ttt.py
offers them too).

The marshalling is native (csrc/binding.cpp): it checks the tensors, makes the
outputs and workspaces that are not given and calls libttt.so. Unlike the
layer's own entry points, these take strided views (innermost dimension
contiguous) and run on the operands' device, whichever device is current, on
its current stream. A `stream` that is given is made the current one for the
call, so what the call allocates belongs to it. Autograd does not see these
calls, an output never requires a gradient: gradients come from the _backward
functions. What a call writes into a tensor of the caller's changes the tensor's
version, as torch's own operators do.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib

_ACT = {"none": _lib.TTT_ACT_NONE, "sigmoid": _lib.TTT_ACT_SIGMOID, "silu": _lib.TTT_ACT_SILU,
        "tanh": _lib.TTT_ACT_TANH}
_CONV_ACT = {"none": _lib.TTT_ACT_NONE, "silu": _lib.TTT_ACT_SILU}
_NORM = {"rms": 0, "layer": 1}


class _Native:
    """The functions of _block.so, which is loaded (after libttt.so) by the first of them."""

    def __getattr__(self, name):
        _lib.load()
        try:
            from . import _block
        except ImportError as e:
            raise ImportError("_block.so is not built; run __graft_entry__.build() or "
                              "python test_sequence_layer_ttt_amd/build.py") from e
        _block.init(_lib.TTTError)
        for k in dir(_block):
            if not k.startswith("_"):
                setattr(self, k, getattr(_block, k))
        return getattr(_block, name)


_native = _Native()


def _choice(table: dict, value, name: str) -> int:
    code = table.get(value)
    if code is None:
        raise ValueError(f"{name} {value!r} is not one of {sorted(table)}")
    return code


def _on(stream, operand, fn, *args):
    """fn(*args) with `stream` (a torch stream or a handle) as the operand's device's current one."""
    if not isinstance(operand, torch.Tensor) or not operand.is_cuda:
        return fn(*args)  # refused there
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(handle, device=operand.device)
    if stream.device != operand.device:
        raise ValueError(f"stream is on {stream.device}, the operands on {operand.device}")
    with torch.cuda.stream(stream):
        return fn(*args)


def _need(name: str, *args: int, pointers=()) -> int:
    for v in args:
        if not -2**31 <= v < 2**31:  # ctypes would cut it to 32 bits
            raise ValueError(f"size {v} is too large")
    n = ctypes.c_size_t(0)
    _lib.check(getattr(_lib.load(), name)(*args, *pointers, ctypes.byref(n)))
    return n.value


# --- short causal convolution ------------------------------------------------


def ttt_conv_forward(x, weight, bias=None, state=None, activation: str = "silu", lens=None, y=None,
                     state_out=None, stream=None):
    """Causal convolution over the last K tokens of each channel, K in 2..4:
    y_t = act(bias + sum_k weight[:, k] x_{t-K+1+k}). x, y [B,L,C] (fp32 or
    bf16, views with a contiguous last dimension allowed), weight [C,K] and
    bias [C] fp32, state [B,K-1,C] the tokens before the first (zeros if
    None), activation "silu" or "none", lens [B] int32 optional lengths.
    Returns (y, state_out); state_out may be `state` itself."""
    args = (x, weight, bias, state, _choice(_CONV_ACT, activation, "activation"), lens, y, state_out)
    if stream is not None:
        return _on(stream, x, _native.conv_forward, *args)
    return _native.conv_forward(*args)


def ttt_conv_step(x, weight, state, bias=None, activation: str = "silu", y=None, stream=None):
    """One token of ttt_conv_forward for each sequence: x [B,C] (a view with a
    contiguous last dimension allowed), state [B,K-1,C] updated in place.
    Returns y [B,C]."""
    args = (x, weight, state, bias, _choice(_CONV_ACT, activation, "activation"), y)
    if stream is not None:
        return _on(stream, x, _native.conv_step, *args)
    return _native.conv_step(*args)


def ttt_conv_backward_workspace(B: int, L: int, C: int, K: int) -> int:
    """Bytes of device workspace ttt_conv_backward needs."""
    return _need("ttt_conv_backward_workspace", B, L, C, K)


def ttt_conv_backward(x, weight, dy, bias=None, state=None, dstate_out=None, activation: str = "silu",
                      lens=None, workspace=None, grads=None, stream=None) -> dict:
    """Gradients of <dy, y> + <dstate_out, state_out> through ttt_conv_forward:
    dx [B,L,C] in x's type, dweight [C,K] fp32, with a bias dbias [C] fp32 and
    with a state dstate [B,K-1,C] in x's type. `grads` may hold the outputs
    (a dict like the one returned; dx may be strided)."""
    args = (x, weight, dy, bias, state, dstate_out, _choice(_CONV_ACT, activation, "activation"), lens,
            workspace, grads)
    if stream is not None:
        return _on(stream, x, _native.conv_backward, *args)
    return _native.conv_backward(*args)


# --- selective state space scan -------------------------------------------------


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
    args = (x, dt, A, B, C, D, dt_bias, state, lens, y, state_out, workspace)
    if stream is not None:
        return _on(stream, x, _native.ssm_forward, *args)
    return _native.ssm_forward(*args)


def ttt_ssm_step(x, dt, A, B, C, state, D=None, dt_bias=None, y=None, stream=None):
    """One token of ttt_ssm_forward for each sequence: x [B,H,P], dt [B,H], B,
    C [B,G,N] (views allowed), state [B,H,N,P] fp32 updated in place. Returns
    y [B,H,P]."""
    args = (x, dt, A, B, C, state, D, dt_bias, y)
    if stream is not None:
        return _on(stream, x, _native.ssm_step, *args)
    return _native.ssm_step(*args)


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
    args = (x, dt, A, B, C, dy, D, dt_bias, state, dstate_out, lens, workspace, grads)
    if stream is not None:
        return _on(stream, x, _native.ssm_backward, *args)
    return _native.ssm_backward(*args)


# --- gated linear recurrence -----------------------------------------------------


def ttt_lru_forward_workspace(B: int, L: int, D: int) -> int:
    """Bytes of device workspace ttt_lru_forward needs."""
    return _need("ttt_lru_forward_workspace", B, L, D)


def ttt_lru_forward(x, r, rate=None, i=None, state=None, lens=None, y=None, state_out=None, workspace=None,
                    stream=None):
    """Gated linear recurrence, a state for each channel: h_t = a_t h_{t-1} +
    s_t sigma(i_t) x_t and y_t = h_t, with log a_t = -rate sigma(r_t), s_t =
    sqrt(1 - a_t^2) or, without a rate, a_t = sigma(r_t), s_t = 1 - a_t (sigma(i)
    is 1 without i). x, r, i, y [B,L,D] in fp32 or bf16 (views with a contiguous
    last dimension allowed, as slices of one projection's output); rate [D] fp32
    >= 0; state, state_out [B,D] fp32; lens [B] int32 optional lengths. Returns
    (y, state_out); state_out may be `state` itself."""
    args = (x, r, rate, i, state, lens, y, state_out, workspace)
    if stream is not None:
        return _on(stream, x, _native.lru_forward, *args)
    return _native.lru_forward(*args)


def ttt_lru_step(x, r, state, rate=None, i=None, y=None, stream=None):
    """One token of ttt_lru_forward for each sequence: x, r, i [B,D] (views with
    a contiguous last dimension allowed), state [B,D] fp32 updated in place.
    Returns y [B,D]."""
    args = (x, r, state, rate, i, y)
    if stream is not None:
        return _on(stream, x, _native.lru_step, *args)
    return _native.lru_step(*args)


def ttt_lru_backward_workspace(B: int, L: int, D: int) -> int:
    """Bytes of device workspace ttt_lru_backward needs."""
    return _need("ttt_lru_backward_workspace", B, L, D)


def ttt_lru_backward(x, r, dy, rate=None, i=None, state=None, dstate_out=None, lens=None, workspace=None, grads=None,
                     stream=None) -> dict:
    """Gradients of <dy, y> + <dstate_out, state_out> through ttt_lru_forward:
    dx, dr and, for those of i, rate and state that are given, di [B,L,D] in x's
    type, drate [D] and dstate [B,D] fp32. `grads` may hold the outputs (a dict
    like the one returned; dx, dr, di may be strided, slices of one buffer too)."""
    args = (x, r, dy, rate, i, state, dstate_out, lens, workspace, grads)
    if stream is not None:
        return _on(stream, x, _native.lru_backward, *args)
    return _native.lru_backward(*args)


# --- products in 8-bit integers ----------------------------------------------------


def ttt_i8_quantize(x, q=None, scale=None, stream=None):
    """Rows of x [...,K] (fp32 or bf16) in 8 bits: scale [...] = max |x| / 127 in
    fp32 and q [...,K] int8, x / scale to the nearest whole number (ties to even).
    A row that holds an infinity or a NaN has a NaN for its scale. For tokens, and
    once for a weight [N,K]. Returns (q, scale)."""
    args = (x, q, scale)
    if stream is not None:
        return _on(stream, x, _native.i8_quantize, *args)
    return _native.i8_quantize(*args)


def _rows(t) -> tuple:
    """Address and row stride of rows of 8-bit values, as the calls take them: a
    dimension of size 1 has no say in the stride."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int8 or t.dim() < 1:
        raise TypeError("rows must be an int8 torch.Tensor")
    stride = next((t.stride(d) for d in range(t.dim() - 2, -1, -1) if t.size(d) != 1), t.size(-1))
    return t.data_ptr() or None, ctypes.byref(ctypes.c_int64(stride))


def _weight(w) -> tuple:
    """Sizes K, N and rows of a weight [N,K]."""
    rows = _rows(w)
    if w.dim() != 2:
        raise ValueError(f"w has shape {tuple(w.shape)}, expected 2 dimensions")
    return w.size(1), w.size(0), rows


def ttt_i8_project_workspace(M: int, x, w) -> int:
    """Bytes of device workspace ttt_i8_project needs for M rows of x and the
    weight w [N,K]: 0 unless M > 64 and rows are not whole 16-byte chunks."""
    K, N, rows = _weight(w)
    return _need("ttt_i8_project_workspace", M, K, N, pointers=(*_rows(x), *rows))


def ttt_i8_project(x, x_scale, w, w_scale, bias=None, dtype=torch.bfloat16, y=None, workspace=None, stream=None):
    """y[...,n] = x_scale[...] w_scale[n] sum_k x[...,k] w[n,k] (+ bias[n]): x
    [...,K] int8 with x_scale [...] fp32 for each row, w [N,K] int8 with w_scale
    [N] and bias [N] fp32; the sum is exact. y [...,N] in `dtype`, bf16 or fp32.
    Rows may be strided (one stride apart)."""
    io = {torch.bfloat16: _lib.TTT_BF16, torch.float32: _lib.TTT_F32}.get(dtype)
    if io is None:
        raise TypeError(f"dtype {dtype} not supported")
    args = (x, x_scale, w, w_scale, bias, io, y, workspace)
    if stream is not None:
        return _on(stream, x, _native.i8_project, *args)
    return _native.i8_project(*args)


def ttt_i8_linear_workspace(M: int, w) -> int:
    """Bytes of device workspace ttt_i8_linear needs for M rows and the weight w
    [N,K] (ttt_qkv_project_i8 for B L rows and theta as [3 H 64, d_model])."""
    K, N, rows = _weight(w)
    return _need("ttt_i8_linear_workspace", M, K, N, pointers=rows)


def ttt_i8_linear(x, w, w_scale, bias=None, y=None, workspace=None, stream=None):
    """ttt_i8_project of x's rows quantised as ttt_i8_quantize does: x [...,K] and
    y [...,N] in fp32 or bf16, w [N,K] int8 with w_scale [N] fp32."""
    args = (x, w, w_scale, bias, y, workspace)
    if stream is not None:
        return _on(stream, x, _native.i8_linear, *args)
    return _native.i8_linear(*args)


def ttt_qkv_project_i8(X, theta, theta_scale, H: int, out=None, workspace=None, stream=None):
    """ttt_qkv_project in 8 bits: X [B,L,d_model] bf16 quantised token by token,
    theta [3,H*64,d_model] int8 with theta_scale [3,H*64] fp32. Returns XQ, XK, XV
    [B,H,L,64] bf16."""
    args = (X, theta, theta_scale, H, None if out is None else tuple(out), workspace)
    if stream is not None:
        return _on(stream, X, _native.qkv_project_i8, *args)
    return _native.qkv_project_i8(*args)


# --- norms, gate and residual between two blocks -------------------------------


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
    args = (resid, y, post_gamma, pre_gamma, gate, scale, post_beta, pre_beta, _choice(_NORM, norm, "norm"),
            _choice(_ACT, gate_act, "gate_act"), eps, lens, resid_out, x)
    if stream is not None:
        return _on(stream, y, _native.block_norm, *args)
    return _native.block_norm(*args)


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
    args = (resid, y, post_gamma, pre_gamma, gate, scale, post_beta, pre_beta, _choice(_NORM, norm, "norm"),
            _choice(_ACT, gate_act, "gate_act"), eps, lens, dresid_out, dx, workspace, grads)
    if stream is not None:
        return _on(stream, y, _native.block_norm_backward, *args)
    return _native.block_norm_backward(*args)
