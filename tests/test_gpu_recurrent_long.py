"""The gated linear recurrence against 64 bits where it is long: prompts by the
longest tiles, gradients over many. Bounds: tests/lru_ref.py's."""
import pytest
import torch

from tests import block_ref as R
from tests import lru_ref as Q
from tests import lru_tiles as T
from tests.test_gpu_recurrent_tiles import _f64, _forward, _inputs
from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("case", T.LONG, ids=str)
def test_forward_by_the_longest_tiles(case):
    """Both decays, with and without input gates, whole tiles and sequences that end
    anywhere in one (NaN behind their ends)."""
    B, L, D, dt, rate, gate, lens = case
    assert T.forward_tokens(B, L, D, dt, gate) == 128
    d = _inputs(B, L, D, dt, rate, gate, lens, 7)
    if lens:
        n = d["lens"].tolist()
        assert 0 in n and 1 in n and L in n and any(1 < v % 128 < 127 for v in n)
    e, keep = _f64(d, B, L)
    y, so = _forward(e["x"], e["r"], e["rate"], e["i"], e["state"], keep)
    b = Q.Bounds(e["x"], e["r"], e["rate"], e["i"], e["state"], e["lens"])
    got, gso = ttt.ttt_lru_forward(d["x"], d["r"], d["rate"], d["i"], d["state"], d["lens"])
    Q.check(got, y, "y", torch.where(b.keep, b.E[:, 1:], 0.0))
    Q.check(gso, so, "state", b.E[:, -1])


def _slow(d):
    """Decays next to 1, by which a tile's borders are felt far away."""
    if d["rate"] is None:
        d["r"] = (d["r"].float() + 6.0).to(d["r"].dtype)
    else:
        d["rate"] = d["rate"] * 0.01
    return d


@pytest.mark.parametrize("case", [(32, 2040, 136, BF, False, False, True), (15, 4400, 136, BF, True, True, True),
                                  (2, 6000, 200, F32, False, True, False), (1, 9001, 33, BF, True, False, False)], ids=str)
def test_forward_of_slow_decays(case):
    B, L, D, dt, rate, gate, lens = case
    d = _slow(_inputs(B, L, D, dt, rate, gate, lens, 8))
    e, keep = _f64(d, B, L)
    y, so = _forward(e["x"], e["r"], e["rate"], e["i"], e["state"], keep)
    b = Q.Bounds(e["x"], e["r"], e["rate"], e["i"], e["state"], e["lens"])
    got, gso = ttt.ttt_lru_forward(d["x"], d["r"], d["rate"], d["i"], d["state"], d["lens"])
    Q.check(got, y, "y", torch.where(b.keep, b.E[:, 1:], 0.0))
    Q.check(gso, so, "state", b.E[:, -1])


# B, L, D, type, rate, gate, lens: 131 to 525 tiles of 16 or 32 tokens, which the carry takes in 16 runs of 9 to 33
# tiles, 8 at a time
CARRIED = [(1, 2100, 24, F32, True, True, False), (3, 2300, 40, BF, True, True, True), (2, 2100, 33, F32, False, True, False),
           (1, 4200, 16, BF, False, False, False), (8, 4200, 12, F32, True, False, True), (1, 8400, 17, F32, True, True, False)]


@pytest.mark.parametrize("slow", [False, True], ids=["fast", "slow"])
@pytest.mark.parametrize("case", CARRIED, ids=str)
def test_backward_over_many_tiles(case, slow):
    B, L, D, dt, rate, gate, lens = case
    d = _inputs(B, L, D, dt, rate, gate, lens, 9)
    d = _slow(d) if slow else d
    e, keep = _f64(d, B, L)
    b = Q.Bounds(e["x"], e["r"], e["rate"], e["i"], e["state"], e["lens"], e["dy"], e["dso"])
    ref = R.gradients(lambda x, r, rate, i, state: _forward(x, r, rate, i, state, keep),
                      {k: e[k] for k in ("x", "r", "rate", "i", "state")}, (e["dy"], e["dso"]))
    got = ttt.ttt_lru_backward(d["x"], d["r"], d["dy"], d["rate"], d["i"], d["state"], d["dso"], d["lens"])
    assert set(got) == {"d" + k for k in ref}
    most = b.gradients()
    for k in got:
        Q.check(got[k], ref[k[1:]], k, most[k])


@pytest.mark.parametrize("B,L,D,dt,gate,lens", [(3, 5000, 40, F32, False, False), (3, 5000, 40, BF, True, True),
                                                (4, 8300, 33, F32, True, True), (32, 4100, 136, BF, False, True),
                                                (1, 40000, 136, BF, False, False)])
def test_values_carried_without_a_rounding(B, L, D, dt, gate, lens):
    """Gates that are open or closed for good (a is 1 or 0): the state is the feature of the
    last token that took one, hundreds of tiles before, and a gradient the sum of whole
    numbers from there on. Every bit is known."""
    g = torch.Generator().manual_seed(10)
    inf = float("inf")
    takes = torch.rand(B, L, D, generator=g) < 1 / 700
    r = torch.where(takes, -inf, inf)
    whole = lambda most, *s: torch.randint(-most, most + 1, s, generator=g).double()
    x, dy, state, dso = whole(100, B, L, D), whole(3, B, L, D), whole(100, B, D), whole(100, B, D)
    n = torch.full((B,), L)
    if lens:
        n = torch.randint(0, L + 1, (B,), generator=g)
        n[0], n[1] = L, 0
    keep = (torch.arange(L)[None] < n[:, None])[..., None]
    h, y = state, torch.zeros(B, L, D, dtype=torch.float64)
    for t in range(L):
        h = torch.where(keep[:, t] & takes[:, t], x[:, t], h)
        y[:, t] = torch.where(keep[:, t], h, 0.0)
    G, dx = dso, torch.zeros(B, L, D, dtype=torch.float64)
    for t in reversed(range(L)):
        at = G + torch.where(keep[:, t], dy[:, t], 0.0)
        take = keep[:, t] & takes[:, t]
        dx[:, t] = torch.where(take, at, 0.0)
        G = torch.where(take, 0.0, at)
    up = lambda v, t=dt: v.to(t).cuda()
    i = up(torch.full((B, L, D), inf)) if gate else None
    lens = n.to(torch.int32).cuda() if lens else None
    gy, gh = ttt.ttt_lru_forward(up(x), up(r), i=i, state=up(state, F32), lens=lens)
    assert torch.equal(gy.cpu(), y.to(dt)) and torch.equal(gh.cpu(), h.float())
    got = ttt.ttt_lru_backward(up(x), up(r), up(dy), i=i, state=up(state, F32), dstate_out=up(dso, F32), lens=lens)
    assert torch.equal(got["dx"].cpu(), dx.float().to(dt)) and torch.equal(got["dstate"].cpu(), G.float())
    for k in ("dr", "di"):
        assert k not in got or not bool(got[k].any())


@pytest.mark.parametrize("rate", [True, False], ids=["rate", "sigma"])
@pytest.mark.parametrize("what", ["x", "state", "r", "i"])
def test_what_is_not_finite_reaches_its_channel_from_its_token_on(what, rate):
    """Infinite features and states and NaN gates: no earlier token, no other channel."""
    B, L, D, t = 2, 700, 16, 333
    d = _inputs(B, L, D, F32, rate, True, False, 11)
    call = lambda: ttt.ttt_lru_forward(d["x"], d["r"], d["rate"], d["i"], d["state"])
    y, so = call()
    if what == "state":
        d["state"][1, 3], t = float("inf"), 0
    else:
        d[what][1, t, 3] = float("inf") if what == "x" else float("nan")
    gy, gs = call()
    bad = ~torch.isfinite(gy)
    assert bool(bad[1, t:, 3].all()) and int(bad.sum()) == L - t
    assert not bool(torch.isfinite(gs[1, 3])) and int((~torch.isfinite(gs)).sum()) == 1
    assert torch.equal(torch.where(bad, y, gy), y)
