"""Python binding of the operators around the layer: the short causal
convolution, the selective state space scan and the block norm, under the C
ABI's names (ttt.py offers them too).

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


def _need(name: str, *args: int) -> int:
    for v in args:
        if not -2**31 <= v < 2**31:  # ctypes would cut it to 32 bits
            raise ValueError(f"size {v} is too large")
    n = ctypes.c_size_t(0)
    _lib.check(getattr(_lib.load(), name)(*args, ctypes.byref(n)))
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
