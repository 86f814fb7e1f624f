"""The gated linear recurrence by tiles of each length, whole ones and cut ones, by
vectors and value by value; 8-bit products of rows that repeat and of odd features.

Bounds: tests/lru_ref.py's; the product's are a rounding each of the integer sum, the
two scales and the bias, and half a step of its type.
"""
import pytest
import torch

from tests import block_ref as R
from tests import lru_ref as Q
from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


def _inputs(B, L, D, dt, rate, gate, lens, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    d = {"x": r(B, L, D).to(dt), "r": r(B, L, D).to(dt), "i": r(B, L, D).to(dt) if gate else None,
         "rate": 0.02 + 2 * torch.rand(D, generator=g) if rate else None, "state": r(B, D), "dy": r(B, L, D).to(dt),
         "dso": r(B, D), "lens": None}
    if lens:  # none, one, the whole, and ends anywhere in a tile
        n = torch.randint(0, L + 1, (B,), generator=g)
        n[0], n[1], n[2] = L, 0, 1
        d["lens"] = n.to(torch.int32)
        for b, t in enumerate(n.tolist()):
            for k in ("x", "r", "i", "dy"):
                if d[k] is not None:
                    d[k][b, t:] = float("nan")
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def _forward(x, r, rate, i, state, keep):
    """The definition, all sequences of a token at once; padded tokens leave the state."""
    a, s = Q.gates(r, rate)
    u = s * x * (1 if i is None else torch.sigmoid(i))
    h, y = state, []
    for t in range(x.shape[1]):
        h = torch.where(keep[:, t], a[:, t] * h + u[:, t], h)
        y.append(torch.where(keep[:, t], h, 0.0))
    return torch.stack(y, 1), h


def _f64(d, B, L):
    e = {k: v if k == "lens" else R.t64(v) for k, v in d.items()}
    keep = R.live(e["lens"], B, L)[1][..., None]
    for k in ("x", "r", "i", "dy"):
        if e[k] is not None:
            e[k] = torch.where(keep, e[k], 0.0)
    return e, keep


FORWARD = [  # tokens of the longest tile that still fills the chip; B, L, D, type, rate, gate, lens
    (64, 32, 1020, 136, BF, True, True, True), (64, 32, 1024, 136, F32, False, True, False),
    (64, 32, 1020, 137, BF, False, True, False), (64, 32, 1020, 137, F32, True, True, True),
    (128, 32, 2040, 136, BF, True, False, False), (128, 32, 1930, 136, F32, False, False, True),
    (128, 15, 4400, 136, BF, True, True, False), (128, 15, 4400, 137, BF, False, True, True),
    (128, 32, 2040, 137, F32, True, False, True),
]


@pytest.mark.parametrize("case", FORWARD, ids=str)
def test_forward_by_each_tile(case):
    tokens, B, L, D, dt, rate, gate, lens = case
    assert B * 2 * -(-L // tokens) >= 1024  # columns by tiles
    d = _inputs(B, L, D, dt, rate, gate, lens, 1)
    e, keep = _f64(d, B, L)
    y, so = _forward(e["x"], e["r"], e["rate"], e["i"], e["state"], keep)
    b = Q.Bounds(e["x"], e["r"], e["rate"], e["i"], e["state"], e["lens"])
    got, gso = ttt.ttt_lru_forward(d["x"], d["r"], d["rate"], d["i"], d["state"], d["lens"])
    Q.check(got, y, "y", torch.where(b.keep, b.E[:, 1:], 0.0))
    Q.check(gso, so, "state", b.E[:, -1])


BACKWARD = [  # B, L, D, type, rate, gate, lens
    (32, 510, 136, BF, True, True, True), (32, 512, 136, F32, False, False, False),
    (32, 510, 137, BF, False, True, False), (32, 510, 137, F32, True, False, True),
    (32, 512, 128, BF, True, True, False), (32, 510, 136, F32, True, True, False),
]


@pytest.mark.parametrize("case", BACKWARD, ids=str)
def test_backward_by_whole_tiles_and_cut_ones(case):
    B, L, D, dt, rate, gate, lens = case
    d = _inputs(B, L, D, dt, rate, gate, lens, 2)
    e, keep = _f64(d, B, L)
    b = Q.Bounds(e["x"], e["r"], e["rate"], e["i"], e["state"], e["lens"], e["dy"], e["dso"])
    ref = R.gradients(lambda x, r, rate, i, state: _forward(x, r, rate, i, state, keep),
                      {k: e[k] for k in ("x", "r", "rate", "i", "state")}, (e["dy"], e["dso"]))
    got = ttt.ttt_lru_backward(d["x"], d["r"], d["dy"], d["rate"], d["i"], d["state"], d["dso"], d["lens"])
    assert set(got) == {"d" + k for k in ref}
    most = b.gradients()
    for k in got:
        Q.check(got[k], ref[k[1:]], k, most[k])


def test_one_workspace_serves_both_kinds_of_tiles():
    """The workspace's size goes by the sizes alone; with input gates the tiles are others."""
    d = _inputs(32, 1024, 136, BF, True, True, False, 3)
    n = ttt.ttt_lru_forward_workspace(32, 1024, 136)
    alone = [ttt.ttt_lru_forward(d["x"], d["r"], d["rate"], i, d["state"])[0] for i in (d["i"], None)]
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for i, y in zip((d["i"], None), alone):
            assert torch.equal(ttt.ttt_lru_forward(d["x"], d["r"], d["rate"], i, d["state"], workspace=ws)[0], y)


def test_features_that_repeat():
    """Rows and tokens of stride 0: one decay gate for all tokens, one token for all sequences."""
    d = _inputs(3, 200, 136, F32, True, True, False, 4)
    r, x = d["r"][:, :1].expand(-1, 200, -1), d["x"][:1].expand(3, -1, -1)
    y, so = ttt.ttt_lru_forward(x, r, d["rate"], d["i"], d["state"])
    y2, so2 = ttt.ttt_lru_forward(x.contiguous(), r.contiguous(), d["rate"], d["i"], d["state"])
    assert torch.equal(y, y2) and torch.equal(so, so2)
    g, g2 = (ttt.ttt_lru_backward(a, c, d["dy"], d["rate"], d["i"], d["state"], d["dso"])
             for a, c in ((x, r), (x.contiguous(), r.contiguous())))
    for k in g:
        assert torch.equal(g[k], g2[k]), k


@pytest.mark.parametrize("M,K,N", [(130, 256, 200), (130, 257, 200), (70, 64, 1), (65, 1, 1), (66, 65536, 17), (40, 48, 70)])
def test_rows_that_repeat(M, K, N):
    """One row of x for all tokens, one of w for all features, and both, as rows of stride 0."""
    g = torch.Generator().manual_seed(5)
    x, w = (torch.randint(-128, 128, (n, K), generator=g).to(I8).cuda() for n in (M, N))
    xs, ws = torch.rand(M, generator=g).cuda() + 0.1, torch.rand(N, generator=g).cuda() + 0.1
    for a, b in ((x[:1].expand(M, -1), w), (x, w[:1].expand(N, -1)), (x[:1].expand(M, -1), w[:1].expand(N, -1)), (x, w)):
        y = ttt.ttt_i8_project(a, xs, b, ws, dtype=F32)
        ref = (a.cpu().double() @ b.cpu().double().t()) * xs.cpu().double()[:, None] * ws.cpu().double()
        R.check(y, ref, "y", 4, ref.abs())


@pytest.mark.parametrize("B,L,dm,H", [(1, 130, 100, 1), (3, 50, 33, 2), (2, 33, 16, 1), (1, 65, 1, 1)])
def test_views_of_many_odd_features(B, L, dm, H):
    g = torch.Generator().manual_seed(6)
    x = torch.randn(B, L, dm, generator=g).to(BF).cuda()
    th = torch.randint(-127, 128, (3, H * 64, dm), generator=g).to(I8).cuda()
    ts = torch.rand(3, H * 64, generator=g).cuda() + 0.1
    out = ttt.ttt_qkv_project_i8(x, th, ts, H)
    q, s = ttt.ttt_i8_quantize(x)
    for k in range(3):
        acc = q.cpu().double().flatten(0, 1) @ th[k].cpu().double().t()
        ref = acc * s.cpu().double().reshape(-1, 1) * ts[k].cpu().double()
        R.check(out[k].transpose(1, 2).reshape(B * L, H * 64), ref, f"view {k}", 4, ref.abs())
