"""The block norm on the GPU against its definition in 64 bits: widths of each
path (one wave a row, a workgroup a row, columns one by one), both norms, every
gate shape and activation, residual types, padded rows that hold NaN, rows of
zeros, strided rows, and the gradients.

Bounds (block_ref.check): a row's sums run over at most 32 columns a thread and
8 joins, the values before them carry a few operations each and the
activations' exp and reciprocal a few steps: 96 half steps of fp32 at the
magnitudes below hold them. A column sum adds n rows along a chain of at most
n / 4 + 64 additions.
"""
import pytest
import torch

from tests import block_ref as R
from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("resid", "y", "post_gamma", "pre_gamma", "gate", "scale", "post_beta", "pre_beta")


def _inputs(B, L, D, dt, rdt, gate, scale, betas, seed, lens=None, wide=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    d = {"resid": (2 * r(B, L, D + wide)).to(rdt).cuda()[..., wide:],
         "y": (0.7 * r(B, L, D + wide)).to(dt).cuda()[..., wide:],
         "post_gamma": (1 + 0.2 * r(D)).cuda(), "pre_gamma": (1 + 0.2 * r(D)).cuda(),
         "gate": {0: lambda: None, 1: lambda: r(D).cuda(), 2: lambda: r(B, D).cuda(),
                  3: lambda: r(B, L, D).to(dt).cuda()}[gate](),
         "scale": (1 + 0.3 * r(D)).cuda() if scale else None,
         "post_beta": (0.3 * r(D)).cuda() if betas else None,
         "pre_beta": (0.3 * r(D)).cuda() if betas else None}
    dro, dx = r(B, L, D).to(rdt).cuda(), r(B, L, D).to(dt).cuda()
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    if lens is not None:
        for b, k in enumerate(lens):
            for t in (d["resid"], d["y"], dro, dx) + ((d["gate"],) if gate == 3 else ()):
                t[b, k:] = float("nan")
    return d, dro, dx, n


CASES = [  # B, L, D, dtype, resid dtype, norm, gate dims, act, scale, betas, lens, wide
    (2, 5, 64, BF, BF, "rms", 0, "none", False, False, None, 0),
    (2, 9, 768, BF, F32, "rms", 3, "sigmoid", True, False, None, 0),
    (3, 7, 768, BF, BF, "layer", 1, "tanh", True, True, [7, 0, 3], 4),
    (2, 6, 2048, BF, F32, "layer", 2, "silu", True, True, [6, 2], 0),
    (1, 1, 1, F32, F32, "rms", 1, "none", True, False, None, 0),
    (2, 3, 37, BF, BF, "layer", 3, "silu", False, True, None, 3),
    (2, 4, 1001, F32, F32, "rms", 2, "tanh", True, False, None, 1),
    (1, 3, 1280, F32, F32, "layer", 3, "none", False, True, None, 0),
    (1, 2, 4100, BF, BF, "rms", 1, "sigmoid", True, False, None, 0),
    (1, 3, 8192, BF, F32, "layer", 3, "tanh", True, True, None, 0),
    (2, 300, 1000, BF, F32, "rms", 3, "silu", True, False, [300, 17], 0),
    (1, 7, 1023, F32, F32, "layer", 1, "sigmoid", True, True, None, 0),
    (2, 290, 2560, BF, BF, "layer", 2, "sigmoid", True, True, [0, 290], 8),
    (1, 600, 4096, BF, F32, "rms", 1, "tanh", False, False, None, 0),
    (1, 5, 4100, F32, F32, "layer", 3, "silu", True, True, None, 0),
    (1, 520, 8192, BF, BF, "rms", 3, "sigmoid", True, False, None, 0),
    (1, 2, 5001, F32, F32, "layer", 0, "none", True, True, None, 0),
    (5, 400, 256, BF, BF, "rms", 2, "sigmoid", True, False, [400, 399, 0, 1, 17], 0),
]


def _run(case, seed):
    B, L, D, dt, rdt, norm, gate, act, scale, betas, lens, wide = case
    d, dro, dx, n = _inputs(B, L, D, dt, rdt, gate, scale, betas, seed, lens, wide)
    ref = {k: R.t64(v) for k, v in d.items()}
    for k in ("resid", "y") + (("gate",) if gate == 3 else ()):
        ref[k] = torch.nan_to_num(ref[k])
    kw = {"norm": norm, "gate_act": act, "eps": 1e-6}
    return d, dro, dx, n, ref, kw


def _call(fn, d, *grads, **kw):
    return fn(d["resid"], d["y"], d["post_gamma"], d["pre_gamma"], *grads, gate=d["gate"], scale=d["scale"],
              post_beta=d["post_beta"], pre_beta=d["pre_beta"], **kw)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    d, _, _, n, ref, kw = _run(case, 1)
    r, x = R.block_norm(**ref, lens=n, **kw)
    gr, gx = _call(ttt.ttt_block_norm, d, lens=n, **kw)
    # magnitudes: |scale resid| + |a n| <= 4 max |r'|; |xhat gamma| + |beta| likewise
    R.check(gr, r, "resid_out", 96, 4 * r.abs().max())
    R.check(gx, x, "x", 96, 4 * x.abs().max())


def _magnitudes(ref, go, kw, n):
    """The largest terms of dresid and dy. A norm's gradient rstd (h - [mean h]
    - hat mean(h hat)) is a difference of terms of up to rstd |h|, |hat| <=
    sqrt(D) and |mean(h hat)| <= max |h|; with one column nothing is left of
    them but eps. rstd is at most that of the row with the least spread."""
    s = 1.0 if ref["scale"] is None else ref["scale"]
    inner = dict(ref, resid=ref["resid"] * s, scale=None)

    def rstd(u):
        u = u - u.mean(-1, keepdim=True) if kw["norm"] == "layer" else u
        return 1 / torch.sqrt((u * u).mean(-1, keepdim=True) + kw["eps"])

    _, keep = R.live(n, *ref["y"].shape[:2])
    keep = keep[..., None]
    most = lambda v: float(torch.where(keep, v, 0.0).abs().max())
    gam = lambda k: 1.0 if ref[k] is None else float(ref[k].abs().max())
    r, _ = R.block_norm(**inner, lens=n, **kw)
    top = most(go[0]) + most(rstd(r)) * most(go[1]) * gam("pre_gamma")
    dr = R.gradients(lambda resid: R.block_norm(**dict(inner, resid=resid), lens=n, **kw),
                     {"resid": inner["resid"]}, go)["resid"]
    a = 1.0 if ref["gate"] is None else float(R.act(ref["gate"], kw["gate_act"]).abs().max())
    return {"resid": 4 * top * max(1.0, float(torch.as_tensor(s).abs().max())),
            "y": 4 * most(rstd(ref["y"])) * max(float(dr.abs().max()), top) * a * gam("post_gamma")}


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    d, dro, dx, n, ref, kw = _run(case, 2)
    B, L = case[0], case[1]
    go = (torch.nan_to_num(R.t64(dro)), torch.nan_to_num(R.t64(dx)))
    want = R.gradients(lambda **v: R.block_norm(**v, lens=n, **kw), ref, go)
    got = _call(ttt.ttt_block_norm_backward, d, dro, dx, lens=n, **kw)
    assert set(got) == {"d" + k for k in want}
    chain = B * L / 4 + 64
    # column sums cancel: their terms' magnitudes are at most max|d| max|hat| a row
    _, keep = R.live(n, B, L)
    rows = max(1, int(keep.sum()))
    mags = _magnitudes(ref, go, kw, n)
    for k, w in want.items():
        g = got["d" + k]
        if k in ("resid", "y") or (k == "gate" and w.dim() == 3):
            R.check(g, w, "d" + k, 192, mags.get(k, 4 * w.abs().max()))
        else:
            term = 4 * max(float(want["resid"].abs().max()), float(go[1].abs().max()), 1.0) * 6
            R.check(g, w, "d" + k, chain + 192, max(float(w.abs().max()), term * rows ** 0.5))


def test_rows_of_zeros_and_of_one_value():
    """sqrt(eps) divides: zero rows stay zero (rms) and constant rows give beta (layer)."""
    D = 128
    z = torch.zeros(1, 3, D, device="cuda", dtype=BF)
    r, x = ttt.ttt_block_norm(z, z)
    assert not bool(r.any()) and not bool(x.any())
    b = torch.full((D,), 0.5, device="cuda")
    c = torch.full((1, 3, D), 3.0, device="cuda", dtype=BF)
    r, x = ttt.ttt_block_norm(z, c, post_beta=b, pre_beta=2 * b, norm="layer")
    assert bool((r == 0.5).all()) and bool((x == 1.0).all())


def test_many_rows_of_one_width_use_every_workgroup():
    """More rows than the grid holds at once: each is its own row's result."""
    d, _, _, _ = _inputs(3, 3000, 512, BF, BF, 1, True, False, 5)
    r, x = _call(ttt.ttt_block_norm, d)
    for b, t in ((0, 0), (1, 1499), (2, 2999)):
        one = dict(d, resid=d["resid"][b:b + 1, t:t + 1].contiguous(), y=d["y"][b:b + 1, t:t + 1].contiguous())
        r1, x1 = _call(ttt.ttt_block_norm, one)
        assert torch.equal(r1[0, 0], r[b, t]) and torch.equal(x1[0, 0], x[b, t])
