"""The state space scan with NaN and infinities in live rows and parameters:
they reach what the definition lets them reach, the same on the matrix cores,
in the vector walk and token by token. Nothing here goes by a tolerance."""
import pytest
import torch

from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
SHAPES = [(2, 200, 3, 64, 64, BF), (1, 70, 2, 24, 40, BF), (1, 90, 2, 33, 20, BF), (2, 256, 96, 64, 32, BF),
          (1, 140, 256, 64, 128, BF), (2, 100, 2, 20, 12, F32), (1, 90, 2, 100, 40, BF)]


def _inputs(B, L, H, P, N, dt, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    d = {"x": r(B, L, H, P).to(dt), "dt": r(B, L, H).to(dt), "A": -torch.rand(H, generator=g) - 0.2,
         "B": r(B, L, 1, N).to(dt), "C": r(B, L, 1, N).to(dt), "D": r(H), "dt_bias": r(H) - 2, "state": r(B, H, N, P)}
    return {k: t.cuda() for k, t in d.items()}


def _forward(d):
    return ttt.ttt_ssm_forward(**d)


def _all_nan(t):
    return bool(torch.isnan(t).all())


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_decay_rate_that_is_not_a_number(shape):
    """A[h] = NaN makes NaN of that head's outputs and state, in a prompt as in
    a single token, and leaves the other heads' bits."""
    d = _inputs(*shape, 1)
    y, so = _forward(d)
    bad = dict(d, A=d["A"].clone())
    bad["A"][1] = NAN
    gy, gs = _forward(bad)
    assert _all_nan(gy[:, :, 1]) and _all_nan(gs[:, 1])
    others = torch.arange(shape[2], device="cuda") != 1
    assert torch.equal(gy[:, :, others], y[:, :, others]) and torch.equal(gs[:, others], so[:, others])
    one = {k: bad[k][:, 0] for k in ("x", "dt", "B", "C")}
    st = d["state"].clone()
    ty = ttt.ttt_ssm_step(**one, A=bad["A"], state=st, D=d["D"], dt_bias=d["dt_bias"])
    assert _all_nan(ty[:, 1]) and _all_nan(st[:, 1])


@pytest.mark.parametrize("value", [NAN, INF], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_step_that_is_not_finite(shape, value):
    """dt at one token: from there on nothing of that head is finite, before it
    and in the other heads every bit stays."""
    d = _inputs(*shape, 2)
    y, _ = _forward(d)
    for t in (0, 37, shape[1] - 1):
        bad = dict(d, dt=d["dt"].clone())
        bad["dt"][0, t, 1] = value
        gy, gs = _forward(bad)
        assert torch.equal(gy[0, :t], y[0, :t]), t
        assert not bool(torch.isfinite(gy[0, t:, 1]).any()) and not bool(torch.isfinite(gs[0, 1]).any())
        gy[0, t:, 1] = y[0, t:, 1]
        assert torch.equal(gy, y)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients_through_a_decay_that_is_not_a_number(shape):
    """g_t = C_t dy_t + a_{t+1} g_{t+1}: a NaN in a decay passes to the gradients
    of every token before it, and to the sums over tokens and heads."""
    d = _inputs(*shape, 3)
    B, L, H = shape[:3]
    dy = torch.randn_like(d["x"])
    bad = dict(d, A=d["A"].clone())
    bad["A"][1] = NAN
    g = ttt.ttt_ssm_backward(**bad, dy=dy)
    assert _all_nan(g["dA"][1]) and _all_nan(g["ddt_bias"][1]) and _all_nan(g["dstate"][:, 1])
    assert _all_nan(g["ddt"][:, :, 1]) and _all_nan(g["dx"][:, :-1, 1]) and _all_nan(g["dB"][:, :-1]) and _all_nan(g["dC"])
    others = torch.arange(H, device="cuda") != 1
    for k in ("dA", "ddt_bias"):
        assert bool(torch.isfinite(g[k][others]).all())
    assert bool(torch.isfinite(g["dx"][:, :, others]).all()) and bool(torch.isfinite(g["ddt"][:, :, others]).all())
    t = L - 2
    bad = dict(d, dt=d["dt"].clone())
    bad["dt"][0, t, 1] = NAN
    g = ttt.ttt_ssm_backward(**bad, dy=dy)
    assert _all_nan(g["dx"][0, :t, 1]) and _all_nan(g["ddt"][0, :, 1]) and _all_nan(g["dB"][0, :t])
    assert _all_nan(g["dstate"][0, 1]) and _all_nan(g["dA"][1]) and _all_nan(g["ddt_bias"][1])


@pytest.mark.parametrize("L", [5, 16, 70])
def test_an_infinite_last_token_of_the_walk(L):
    """The rows staged behind a walk's last token add nothing to the state, also
    where that token's values are infinite: the prompt's state is the one that
    single tokens give."""
    d = _inputs(2, L, 2, 20, 12, F32, 4)
    d["x"][0, L - 1, 1, 3] = INF
    st = d["state"].clone()
    for t in range(L):
        one = {k: d[k][:, t] for k in ("x", "dt", "B", "C")}
        ttt.ttt_ssm_step(**one, A=d["A"], state=st, D=d["D"], dt_bias=d["dt_bias"])
    _, so = _forward(d)
    want = INF * d["B"][0, L - 1, 0].sign()
    assert torch.equal(st[0, 1, :, 3], want) and torch.equal(so[0, 1, :, 3], want)
    so[0, 1, :, 3] = 0
    assert bool(torch.isfinite(so).all())


@pytest.mark.parametrize("value", [NAN, INF, -INF], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_row_that_is_not_finite(shape, value):
    """A value of x, B or C that is not finite reaches what its token and those
    behind it make of it: x its own feature, B the whole head, C its token. The
    outputs before it, of a prompt as of single tokens, keep their bits."""
    d = _inputs(*shape, 5)
    B, L, H, P, N, _ = shape
    y, so = _forward(d)
    for t in (0, 13, 38, 64, L - 1):
        if t >= L:
            continue
        for k in ("x", "B", "C"):
            bad = dict(d, **{k: d[k].clone()})
            i = (7 * t + 3) % (P if k == "x" else N)
            bad[k][0, t, 0, i] = value
            gy, gs = _forward(bad)
            hit = torch.zeros_like(y, dtype=torch.bool)
            if k == "x":
                hit[0, t:, 0, i] = True
            else:
                hit[0, t:L if k == "B" else t + 1] = True
            assert not bool(torch.isfinite(gy[hit]).any()), (k, t)
            assert torch.equal(gy[~hit], y[~hit]), (k, t)
            where = torch.zeros_like(so, dtype=torch.bool)
            if k == "x":
                where[0, 0, :, i] = True
            elif k == "B":
                where[0, :, i] = True
            assert not bool(torch.isfinite(gs[where]).any()), (k, t)
            assert torch.equal(gs[~where], so[~where]), (k, t)


def test_rows_of_which_many_are_not_finite():
    """Several features and tokens of one chunk, found by different waves, and a
    chunk behind them that is finite again."""
    B, L, H, P, N, dt = 1, 200, 768, 64, 16, BF
    d = _inputs(B, L, H, P, N, dt, 6)
    y, _ = _forward(d)
    bad = dict(d, x=d["x"].clone())
    at = [(70, 3, NAN), (70, 60, INF), (101, 3, INF), (66, 33, -INF), (127, 0, NAN), (64, 17, INF), (150, 5, NAN)]
    hit = torch.zeros_like(y, dtype=torch.bool)
    for t, p, v in at:
        bad["x"][0, t, 5, p] = v
        hit[0, t:, 5, p] = True
    gy, _ = _forward(bad)
    assert not bool(torch.isfinite(gy[hit]).any()) and torch.equal(gy[~hit], y[~hit])
