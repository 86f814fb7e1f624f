"""The state space scan and its gradients in 64 bits, token by token with every
sequence and head at once, on the device of its inputs: for sizes at which
torch's differentiation of block_ref.scan is too slow. Along with the gradients
it gives the sums that their bounds go by. tests/test_scan_ref.py holds it to
block_ref.scan, to torch's differentiation and to differences."""
from __future__ import annotations

import torch

KEYS = ("x", "dt", "A", "Bm", "Cm", "D", "dt_bias", "state")
CHUNK = 64  # tokens of a chunk of the matrix-core kernels


def t64(v):
    return None if v is None else v.detach().double()


def absolute(v):
    """The same scan of the terms' magnitudes."""
    return {k: t if t is None or k in ("dt", "A", "dt_bias") else t.abs() for k, t in v.items()}


def scan(v, n=None, dy=None, dso=None):
    """v: 64-bit operands by the names of KEYS (D, dt_bias, state may be None);
    n: [B] lengths or None. {"y", "state_out"}, and with dy [B,L,H,P] and dso
    [B,H,N,P] the gradients by their names and, for the bounds of the decay's,
      q    [B,L,H] what passes from the tokens before t to those from t on
      row, col     the parts of q that end (begin) at a token, its own term excluded
      ends [B,K,H] what a chunk's borders pass: q at its start
      final [B,H]  the last state times its gradient
      over [B,K,H] the state before a chunk times the gradient behind it, undecayed."""
    x, z, A, Bm, Cm, D, bias, state = (v[k] for k in KEYS)
    B, L, H, P = x.shape
    G, N = Bm.shape[2:]
    head = torch.arange(H, device=x.device) // (H // G)
    n = torch.full((B,), L, device=x.device) if n is None else n.long().clamp(0, L)
    live = torch.arange(L, device=x.device)[None] < n[:, None]
    keep = lambda t: torch.where(live.reshape(B, L, *[1] * (t.dim() - 2)), t, 0.0)
    z = z if bias is None else z + bias
    x, Bm, Cm, z = keep(x), keep(Bm), keep(Cm), keep(z)
    d = keep(torch.logaddexp(z, torch.zeros_like(z)))
    a, u = torch.exp(d * A), d[..., None] * x
    h = x.new_zeros(B, H, N, P) if state is None else state
    hs, y = [h], torch.zeros_like(x)
    for t in range(L):
        h = a[:, t, :, None, None] * h + Bm[:, t, head, :, None] * u[:, t, :, None, :]
        y[:, t] = (Cm[:, t, head, :, None] * h).sum(2)
        if dy is None:
            hs = [h]
        else:
            hs.append(h)
    out = {"y": keep(y if D is None else y + D[:, None] * x), "state_out": h}
    if dy is None:
        return out
    dy = keep(dy)
    K = -(-L // CHUNK)
    r = torch.zeros_like(h) if dso is None else dso  # the gradient of the state behind token t
    du, q, row, col = torch.zeros_like(x), torch.zeros_like(d), torch.zeros_like(d), torch.zeros_like(d)
    dBh, dCh = x.new_zeros(B, L, H, N), x.new_zeros(B, L, H, N)
    ends, over = x.new_zeros(B, K, H), x.new_zeros(B, K, H)
    behind = r
    for t in reversed(range(L)):
        before, dec = hs[t], a[:, t, :, None, None]
        if t % CHUNK == CHUNK - 1 or t == L - 1:
            behind = r
        Bt, Ct = Bm[:, t, head], Cm[:, t, head]
        col[:, t] = (Bt * (r * u[:, t, :, None, :]).sum(-1)).sum(-1)
        row[:, t] = (Ct * (dec * before * dy[:, t, :, None, :]).sum(-1)).sum(-1)
        g = r + Ct[..., None] * dy[:, t, :, None, :]
        du[:, t] = (Bt[..., None] * g).sum(2)
        dBh[:, t] = (g * u[:, t, :, None, :]).sum(-1)
        dCh[:, t] = (hs[t + 1] * dy[:, t, :, None, :]).sum(-1)
        q[:, t] = (g * dec * before).sum((-1, -2))
        r = dec * g
        if t % CHUNK == 0:
            ends[:, t // CHUNK] = q[:, t]
            over[:, t // CHUNK] = (before * behind).sum((-1, -2))
    xdu, sig = (x * du).sum(-1), keep(1 / (1 + torch.exp(-z)))
    ddt = (q * A + xdu) * sig
    per_group = lambda t: keep(t.unflatten(2, (G, H // G)).sum(3))
    out.update(dx=keep(d[..., None] * du + (0 if D is None else D[:, None] * dy)), ddt=ddt, dA=(q * d).sum((0, 1)),
               dB=per_group(dBh), dC=per_group(dCh), q=keep(q), row=row, col=col, ends=ends, over=over,
               final=(hs[L] * (torch.zeros_like(h) if dso is None else dso)).sum((-1, -2)), step=d, sig=sig,
               xdu=keep(xdu))
    if D is not None:
        out["dD"] = (dy * x).sum((0, 1, 3))
    if bias is not None:
        out["ddt_bias"] = ddt.sum((0, 1))
    if state is not None:
        out["dstate"] = r
    return out


def decay_sums(m, ops):
    """What the decay's gradient of a token is summed from, for a scan `m` of
    magnitudes: the parts of the tokens up to 64 behind it (a running sum), and
    what the borders of its segment pass, at most four chunks either way, each
    taken twice and once more as the product of a state and its gradient. A
    chunk whose decay is below 2^-24 counts as passing nothing: 2^-24 of
    `over`, here in units of the caller's `ops` half steps of fp32."""
    L, K = m["q"].shape[1], m["ends"].shape[1]
    out = torch.empty_like(m["q"])
    part = m["row"] + m["col"]
    for t in range(L):
        k = t // CHUNK
        near = slice(max(0, k - 4), min(K, k + 5))
        last = m["q"][:, min(t + CHUNK, L - 1)]
        out[:, t] = (m["q"][:, t] + last + part[:, t:t + CHUNK].sum(1) + 3 * m["ends"][:, near].sum(1)
                     + 3 * m["final"] + m["over"][:, near].sum(1) / ops)
    return out
