"""Plain definitions, in 64 bits on the CPU, of the operators around the layer,
and the bound that a result in fp32 or bf16 has to keep to. Gradients come from
torch's differentiation of these definitions."""
from __future__ import annotations

import torch

F64 = torch.float64
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def t64(t):
    return None if t is None else t.detach().cpu().to(F64)


def live(lens, B, L):
    n = torch.full((B,), L) if lens is None else lens.cpu().long().clamp(0, L)
    return n, torch.arange(L)[None] < n[:, None]  # [B], [B,L]


def conv(x, w, bias, state, act, lens):
    """(y, state_out) of the causal convolution, sequence by sequence."""
    B, L, C = x.shape
    K = w.shape[1]
    n, _ = live(lens, B, L)
    y, so = [], []
    for b in range(B):
        full = torch.cat([x.new_zeros(K - 1, C) if state is None else state[b], x[b, :n[b]]])
        z = sum(w[:, k] * full[k:k + n[b]] for k in range(K))
        if bias is not None:
            z = z + bias
        if act == "silu":
            z = z / (1 + torch.exp(-z))
        y.append(torch.cat([z, x.new_zeros(L - int(n[b]), C)]))
        so.append(full[n[b]:])
    return torch.stack(y), torch.stack(so)


def scan(x, dt, A, Bm, Cm, D, dt_bias, state, lens, dt_in=None):
    """(y, state_out) of the state space scan, token by token. dt_in: a second
    dt for the inputs alone, to tell its two gradients apart."""
    B, L, H, P = x.shape
    G, N = Bm.shape[2:]
    n, _ = live(lens, B, L)
    head = torch.arange(H) // (H // G)
    y, so = [], []
    for b in range(B):
        h = x.new_zeros(H, N, P) if state is None else state[b]
        rows = []
        for t in range(int(n[b])):
            z = dt[b, t] + (0 if dt_bias is None else dt_bias)
            d = torch.logaddexp(z, torch.zeros_like(z))
            a = torch.exp(d * A)
            if dt_in is not None:
                z = dt_in[b, t] + (0 if dt_bias is None else dt_bias)
                d = torch.logaddexp(z, torch.zeros_like(z))
            h = a[:, None, None] * h + Bm[b, t][head][:, :, None] * (d[:, None] * x[b, t])[:, None, :]
            row = (Cm[b, t][head][:, :, None] * h).sum(1)
            rows.append(row if D is None else row + D[:, None] * x[b, t])
        rows += [x.new_zeros(H, P)] * (L - int(n[b]))
        y.append(torch.stack(rows) if rows else x.new_zeros(0, H, P))
        so.append(h)
    return torch.stack(y), torch.stack(so)


def act(v, name):
    return {"none": lambda: v, "sigmoid": lambda: 1 / (1 + torch.exp(-v)),
            "silu": lambda: v / (1 + torch.exp(-v)), "tanh": lambda: torch.tanh(v)}[name]()


def block_norm(resid, y, post_gamma, pre_gamma, gate, scale, post_beta, pre_beta, norm, gate_act, eps, lens):
    """(resid_out, x) of the block norm; padded rows are replaced before they are used."""
    B, L, _ = y.shape
    _, keep = live(lens, B, L)
    keep = keep[..., None]
    resid, y = torch.where(keep, resid, 0.0), torch.where(keep, y, 0.0)

    def unit(u, gamma, beta):
        if norm == "layer":
            u = u - u.mean(-1, keepdim=True)
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps)
        u = u if gamma is None else u * gamma
        return u if beta is None else u + beta

    n = unit(y, post_gamma, post_beta)
    if gate is not None:
        g = torch.where(keep, gate, 0.0) if gate.dim() == 3 else gate[:, None] if gate.dim() == 2 else gate
        n = n * act(g, gate_act)
    r = (resid if scale is None else resid * scale) + n
    x = unit(r, pre_gamma, pre_beta)
    return torch.where(keep, r, 0.0), torch.where(keep, x, 0.0)


def gradients(fn, leaves: dict, outs_grad) -> dict:
    """d<fn(leaves), outs_grad> for each leaf that is not None."""
    leaf = {k: v.clone().requires_grad_(True) for k, v in leaves.items() if v is not None}
    outs = fn(**{k: leaf.get(k) for k in leaves})
    loss = sum((o * g).sum() for o, g in zip(outs, outs_grad) if g is not None)
    g = torch.autograd.grad(loss, list(leaf.values()), allow_unused=True)
    return {k: torch.zeros_like(v) if d is None else d for (k, v), d in zip(leaf.items(), g)}


def check(got, ref, name, ops, mag=None, roundings=0.0):
    """|got - ref| <= half a step of got's type at |ref|, plus `ops` half steps
    of fp32 at `mag` (the largest |ref| unless given: the sum of the terms'
    magnitudes where terms cancel), plus `roundings` half steps of bf16 at
    `mag` (operands that a matrix product takes rounded)."""
    got, dt = got.detach().cpu().to(F64), got.dtype
    ref = ref.detach()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if ref.numel() == 0:
        return
    assert torch.isfinite(got).all(), f"{name} is not finite"
    m = ref.abs().max() if mag is None else mag
    noise = (ops * 2.0 ** -24 + roundings * 2.0 ** -8) * m
    bound = HALF_STEP[dt] * (ref.abs() + noise) + noise + 1e-30
    worst = float(((got - ref).abs() / bound).max())
    print(f"[block] {name}: {worst:.2f} of the bound", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bound"
