"""Plain definition, in 64 bits on the CPU, of the gated linear recurrence, token
by token, and how far fp32 arithmetic may be from it.

Bounds, in half steps of fp32 (h = 2^-24), with R the largest |r|, |i| and Z the
largest rate. An exponential of argument v is off by 2 |v| + 2 (the argument's
product, the instruction), a sigmoid by 2 R + 8 with its sum, reciprocal and
product; z = -rate sigma(r) by ez = 2 R + 9. Where |z| < 0.1, 1 - a is off by ez
and 6 roundings of its series; elsewhere by what e^z is off by, at most 2.8 +
0.37 ez, over 1 - a > 0.095: ez + 32 holds both. s, its root, is off by half of
that and 4. So u = s sigma(i) x is off by EU = 16 + ez / 2 + 4 + 2 R + 8 + 3, a by
EA = 2 R + 14 of 1 (of a by EAR = 2 + Z (ez + 2) + 2 R + 14), three roundings of a
product of decays and of the state's sum with it. The state's error then follows
the recurrence itself, E_t = a_t E_{t-1} + h (EA M_{t-1} + EU |u_t| + 2 M_t), M
the recurrence over |u|; the gradient's likewise, backwards.
"""
from __future__ import annotations

import torch

from tests.block_ref import F64, HALF_STEP, live

H = 2.0 ** -24


def gates(r, rate):
    """a, s of every token"""
    if rate is None:
        return torch.sigmoid(r), torch.sigmoid(-r)
    z = -rate * torch.sigmoid(r)
    return torch.exp(z), torch.sqrt(-torch.expm1(2 * z))


def forward(x, r, rate, i, state, lens):
    """(y, state_out), sequence by sequence and token by token."""
    B, L, D = x.shape
    n, _ = live(lens, B, L)
    y, so = [], []
    for b in range(B):
        h = x.new_zeros(D) if state is None else state[b]
        rows = []
        for t in range(int(n[b])):
            a, s = gates(r[b, t], rate)
            u = s * x[b, t] * (1 if i is None else torch.sigmoid(i[b, t]))
            h = a * h + u
            rows.append(h)
        rows += [x.new_zeros(D)] * (L - int(n[b]))
        y.append(torch.stack(rows) if rows else x.new_zeros(0, D))
        so.append(h)
    return torch.stack(y), torch.stack(so)


class Bounds:
    """M, E of the state before and after each token, MG, EG of the gradient, and the constants."""

    def __init__(self, x, r, rate, i, state, lens, dy=None, dso=None):
        B, L, D = x.shape
        n, keep = live(lens, B, L)
        self.keep = keep[..., None]
        zero = torch.zeros((), dtype=F64)
        x, r = (torch.where(self.keep, v, zero) for v in (x, r))
        i = None if i is None else torch.where(self.keep, i, zero)
        R = max([float(v.abs().max()) if v.numel() else 0.0 for v in (r, i) if v is not None])
        Z = 0.0 if rate is None else float(rate.max())
        ez = 2 * R + 9
        self.EU = 16 + ez / 2 + 4 + 2 * R + 8 + 3
        self.EA, self.ES = 2 * R + 14, 2 * R + 10
        self.EAR = 2 + Z * (ez + 2) + self.EA
        self.a, self.s = gates(r, rate)
        self.g = torch.sigmoid(r)
        self.e = torch.ones_like(x) if i is None else torch.sigmoid(i)
        self.v = self.e * x
        a, u = torch.where(self.keep, self.a, 1.0), torch.where(self.keep, (self.s * self.v).abs(), 0.0)
        M = torch.zeros(B, D, dtype=F64) if state is None else state.abs()
        E = torch.zeros(B, D, dtype=F64)
        Ms, Es = [M], [E]
        for t in range(L):
            E = a[:, t] * E + H * torch.where(self.keep[:, t], self.EA * M + self.EU * u[:, t], 0.0)
            M = a[:, t] * M + u[:, t]
            E = E + H * 2 * M
            Ms.append(M)
            Es.append(E)
        self.M, self.E = torch.stack(Ms, 1), torch.stack(Es, 1)  # [B,L+1,D]
        if dy is None:
            return
        G = torch.zeros(B, D, dtype=F64) if dso is None else dso.abs()
        E = torch.zeros(B, D, dtype=F64)
        dy = torch.where(self.keep, dy, zero).abs()
        Gs, Es = [], []
        for t in reversed(range(L)):
            G = G + dy[:, t]
            E = E + H * 2 * G
            Gs.append(G)  # of this token's h
            Es.append(E)
            E = a[:, t] * E + H * torch.where(self.keep[:, t], self.EA * G, 0.0)
            G = a[:, t] * G
        self.K, self.EK = G, E  # what flows into the state before the first token
        self.G = torch.stack(Gs[::-1], 1) if Gs else torch.zeros(B, 0, D, dtype=F64)
        self.EG = torch.stack(Es[::-1], 1) if Es else self.G
        self.rate = rate

    def gradients(self):
        """{name: the most that fp32 arithmetic may be off}"""
        a, s, e, v, G, EG = self.a, self.s, self.e, self.v.abs(), self.G, self.EG
        M, EM = self.M[:, :-1], self.E[:, :-1]
        w = torch.where(self.keep, 1.0, 0.0).to(F64)
        out = {"dx": w * s * e * (EG + H * (self.EU + self.ES) * G),
               "di": w * s * v * (1 - e) * (EG + H * (self.EU + 3 * self.ES) * G)}
        slope = a if self.rate is None else torch.where(s > 0, a * a / torch.where(s > 0, s, 1.0), 0.0)
        mag = a * M + v * slope
        l = EG * mag + G * (a * EM + H * (self.EAR * a * M + (2 * self.EAR + 2 * self.EU) * v * slope + 4 * mag))
        lm = G * mag
        if self.rate is None:
            out["dr"] = w * s * (l + H * 2 * self.ES * lm)
        else:
            q = self.g * (1 - self.g) * self.rate
            out["dr"] = w * q * (l + H * (3 * self.ES + 4) * lm)
            chain = 100 + lm.shape[0] * lm.shape[1] / 1000
            out["drate"] = (w * self.g * (l + H * (self.ES + chain) * lm)).sum((0, 1))
        out["dstate"] = self.EK + H * self.EA * self.K
        return out


def check(got, ref, name, bound):
    """|got - ref| <= half a step of got's type at what fp32 arithmetic may give, plus its own bound."""
    got, dt = got.detach().cpu().to(F64), got.dtype
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if ref.numel() == 0:
        return
    assert torch.isfinite(got).all(), f"{name} is not finite"
    most = HALF_STEP[dt] * (ref.detach().abs() + bound) + bound + 1e-30
    worst = float(((got - ref.detach()).abs() / most).max())
    print(f"[lru] {name}: {worst:.2f} of the bound", flush=True)
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bound"
