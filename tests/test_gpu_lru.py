"""The gated linear recurrence on the GPU against its definition in 64 bits: both
decays, with and without an input gate, lengths of zero and one and at the
tiles' borders, ragged batches, strided slices, single tokens after a prompt,
and its gradients against the formula's and against differences. Bounds:
lru_ref.
"""
import pytest
import torch

from tests import block_ref as R
from tests import lru_ref as Q
from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _inputs(B, L, D, dt, seed=0, rate=True, gate=True, state=True, lens=None, wide=0, slow=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    xri = r(B, L, (2 + gate) * D + wide).to(dt).cuda()[..., wide:]
    base = 0.02 if slow else 1.0
    return {"x": xri[..., :D], "r": xri[..., D:2 * D], "i": xri[..., 2 * D:] if gate else None,
            "rate": (base * (0.02 + 2 * torch.rand(D, generator=g))).cuda() if rate else None,
            "state": r(B, D).cuda() if state else None, "dy": r(B, L, D).to(dt).cuda(), "dso": r(B, D).cuda(),
            "lens": None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()}


def _poison(d):
    """NaN in every padded row: it must not be read."""
    if d["lens"] is not None:
        for b, n in enumerate(d["lens"].tolist()):
            for k in ("x", "r", "i", "dy"):
                if d[k] is not None:
                    d[k][b, n:] = float("nan")
    return d


def _f64(d):
    return {k: R.t64(v) if k != "lens" else v for k, v in d.items()}


CASES = [  # B, L, D, dtype, rate, gate, state, lens, wide
    (2, 37, 64, BF, True, True, True, None, 8),
    (1, 1, 8, BF, True, False, False, None, 0),
    (3, 2, 24, F32, False, True, True, None, 4),
    (2, 19, 7, F32, True, True, True, None, 1),
    (2, 64, 16, BF, False, False, True, None, 0),
    (2, 65, 16, F32, True, True, True, None, 0),
    (1, 128, 136, BF, True, True, False, None, 0),
    (1, 129, 136, BF, False, True, True, None, 0),
    (4, 300, 40, BF, True, True, True, [0, 1, 300, 177], 3),
    (3, 200, 33, F32, False, False, True, [200, 2, 0], 0),
    (3, 257, 130, BF, True, False, False, [129, 128, 257], 2),
    (2, 1300, 24, F32, True, True, True, [1300, 1111], 0),
    (2, 0, 16, BF, True, True, True, None, 0),
]


def _args(d):
    return (d["x"], d["r"]), {"rate": d["rate"], "i": d["i"], "state": d["state"], "lens": d["lens"]}


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    B, L, D, dt, rate, gate, state, lens, wide = case
    d = _poison(_inputs(B, L, D, dt, 1, rate, gate, state, lens, wide))
    e = _f64(d)
    y, so = Q.forward(e["x"], e["r"], e["rate"], e["i"], e["state"], e["lens"])
    b = Q.Bounds(e["x"], e["r"], e["rate"], e["i"], e["state"], e["lens"])
    a, kw = _args(d)
    got, gso = ttt.ttt_lru_forward(*a, **kw)
    Q.check(got, y, "y", torch.where(b.keep, b.E[:, 1:], 0.0))
    Q.check(gso, so, "state", b.E[:, -1])
    # the state may be replaced where it stands
    if state:
        st = d["state"].clone()
        got2, st2 = ttt.ttt_lru_forward(*a, **{**kw, "state": st}, state_out=st)
        assert st2.data_ptr() == st.data_ptr() and torch.equal(st, gso) and torch.equal(got2, got)


@pytest.mark.parametrize("rate", [True, False])
def test_slow_decays_at_length(rate):
    """Decays next to 1, whose states hold thousands of tokens."""
    d = _inputs(1, 4000, 32, F32, 2, rate, True, slow=True)
    if not rate:
        d["r"] += 6.0
    e = _f64(d)
    y, so = Q.forward(e["x"], e["r"], e["rate"], e["i"], e["state"], None)
    b = Q.Bounds(e["x"], e["r"], e["rate"], e["i"], e["state"], None)
    a, kw = _args(d)
    got, gso = ttt.ttt_lru_forward(*a, **kw)
    Q.check(got, y, "y", b.E[:, 1:])
    Q.check(gso, so, "state", b.E[:, -1])


@pytest.mark.parametrize("dt,D,wide,rate,gate", [(BF, 64, 0, True, True), (F32, 33, 5, False, True), (BF, 17, 3, True, False),
                                                 (F32, 768, 4, True, True), (BF, 2048, 8, False, False)])
def test_single_tokens_continue_a_prompt(dt, D, wide, rate, gate):
    """Steps after a prompt: each within its bound of the whole prompt's definition."""
    B, L, T = 3, 9, 6
    d = _inputs(B, L + T, D, dt, 3, rate, gate, wide=wide)
    e = _f64(d)
    y, so = Q.forward(e["x"], e["r"], e["rate"], e["i"], e["state"], None)
    b = Q.Bounds(e["x"], e["r"], e["rate"], e["i"], e["state"], None)
    cut = lambda v, s: None if v is None else v[:, s]
    _, st = ttt.ttt_lru_forward(d["x"][:, :L], d["r"][:, :L], d["rate"], cut(d["i"], slice(L)), d["state"])
    for t in range(L, L + T):
        got = ttt.ttt_lru_step(d["x"][:, t], d["r"][:, t], st, d["rate"], cut(d["i"], t))
        Q.check(got, y[:, t], f"y of token {t}", b.E[:, t + 1])
    Q.check(st, so, "state", b.E[:, -1])


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    B, L, D, dt, rate, gate, state, lens, wide = case
    d = _poison(_inputs(B, L, D, dt, 4, rate, gate, state, lens, wide))
    e = _f64(d)
    b = Q.Bounds(e["x"], e["r"], e["rate"], e["i"], e["state"], e["lens"], e["dy"], e["dso"])
    clean = {k: None if e[k] is None else torch.where(b.keep, e[k], 0.0) for k in ("x", "r", "i", "dy")}
    ref = R.gradients(lambda x, r, rate, i, state: Q.forward(x, r, rate, i, state, e["lens"]),
                      {"x": clean["x"], "r": clean["r"], "rate": e["rate"], "i": clean["i"], "state": e["state"]},
                      (clean["dy"], e["dso"]))
    got = ttt.ttt_lru_backward(d["x"], d["r"], d["dy"], d["rate"], d["i"], d["state"], d["dso"], d["lens"])
    assert set(got) == {"d" + k for k in ref}
    most = b.gradients()
    for k in got:
        Q.check(got[k], ref[k[1:]], k, most[k])


def test_gradients_against_differences():
    """The loss moved by small steps of each input, in 64 bits, along random directions."""
    B, L, D = 2, 70, 9
    d = _inputs(B, L, D, F32, 5)
    e = _f64(d)
    got = ttt.ttt_lru_backward(d["x"], d["r"], d["dy"], d["rate"], d["i"], d["state"], d["dso"])
    args = {k: e[k] for k in ("x", "r", "rate", "i", "state")}

    def loss(**kw):
        y, so = Q.forward(**{**args, **kw}, lens=None)
        return float((y * e["dy"]).sum() + (so * e["dso"]).sum())

    most = Q.Bounds(e["x"], e["r"], e["rate"], e["i"], e["state"], None, e["dy"], e["dso"]).gradients()
    g = torch.Generator().manual_seed(6)
    for k in args:
        way = torch.randn(args[k].shape, generator=g, dtype=torch.float64)
        step = 1e-5
        diff = (loss(**{k: args[k] + step * way}) - loss(**{k: args[k] - step * way})) / (2 * step)
        off = abs(float((got["d" + k].cpu().double() * way).sum()) - diff)
        # the kernel's own bound, and a third derivative of at most 1e3 |way| steps
        near = float((most["d" + k] * way.abs()).sum()) + 1e-6 * float((got["d" + k].cpu().abs().double() * way.abs()).sum()) + 1e-6
        assert off <= near, (k, off, near)


def test_gradients_into_slices_of_one_buffer():
    """dx, dr and di may be slices of one wider buffer, whose other columns stay."""
    D = 24
    d = _inputs(2, 150, D, BF, 7)
    ref = ttt.ttt_lru_backward(d["x"], d["r"], d["dy"], d["rate"], d["i"], d["state"], d["dso"])
    wide = torch.full((2, 150, 3 * D + 16), 7.0, dtype=BF, device="cuda")
    g = {k: torch.empty_like(v) for k, v in ref.items()}
    for n, k in enumerate(("dx", "dr", "di")):
        g[k] = wide[..., 8 + n * D:8 + (n + 1) * D]
    ttt.ttt_lru_backward(d["x"], d["r"], d["dy"], d["rate"], d["i"], d["state"], d["dso"], grads=g)
    assert all(torch.equal(g[k], ref[k]) for k in ref)
    assert bool((wide[..., :8] == 7).all()) and bool((wide[..., 8 + 3 * D:] == 7).all())


def test_outputs_into_a_slice():
    D = 40
    d = _inputs(2, 33, D, F32, 8)
    a, kw = _args(d)
    ref, _ = ttt.ttt_lru_forward(*a, **kw)
    wide = torch.full((2, 33, D + 9), 7.0, device="cuda")
    ttt.ttt_lru_forward(*a, **kw, y=wide[..., 5:5 + D])
    assert torch.allclose(wide[..., 5:5 + D], ref, rtol=1e-6, atol=1e-6)  # read one by one here
    assert bool((wide[..., :5] == 7).all()) and bool((wide[..., 5 + D:] == 7).all())


def test_gates_at_their_ends():
    """r of infinity, closed and open, and i of infinity: the definition's limits, without NaN."""
    inf = float("inf")
    x = torch.ones(1, 6, 8, device="cuda")
    r = torch.tensor([0.0, -inf, inf, -200.0, 200.0, 0.0], device="cuda")[None, :, None].repeat(1, 1, 8)
    i = torch.tensor([0.0, 0.0, -inf, inf, 100.0, -100.0], device="cuda")[None, :, None].repeat(1, 1, 8)
    rate = torch.full((8,), 0.5, device="cuda")
    for q in (rate, None):
        y, so = ttt.ttt_lru_forward(x, r, rate=q, i=i)
        ry, rso = Q.forward(R.t64(x), R.t64(r), R.t64(q), R.t64(i), None, None)
        assert torch.allclose(R.t64(y), ry, rtol=1e-5, atol=1e-7) and torch.allclose(R.t64(so), rso, rtol=1e-5, atol=1e-7)
        g = ttt.ttt_lru_backward(x, r, torch.ones_like(x), rate=q, i=i)
        assert all(bool(torch.isfinite(v).all()) for v in g.values())


@pytest.mark.parametrize("L,t", [(5, 2), (300, 130)])
def test_a_nan_stays_behind_its_token_and_in_its_channel(L, t):
    d = _inputs(2, L, 16, BF, 9)
    a, kw = _args(d)
    ref, _ = ttt.ttt_lru_forward(*a, **kw)
    d["x"][1, t, 3] = float("nan")
    y, so = ttt.ttt_lru_forward(*a, **kw)
    bad = torch.isnan(y)
    assert bool(bad[1, t:, 3].all()) and int(bad.sum()) == L - t and bool(torch.isnan(so[1, 3])) and int(torch.isnan(so).sum()) == 1
    assert torch.equal(torch.where(bad, ref, y), ref)


def test_the_same_bits_every_time():
    d = _inputs(2, 1000, 200, BF, 10)
    a, kw = _args(d)
    first = ttt.ttt_lru_forward(*a, **kw)
    g = ttt.ttt_lru_backward(d["x"], d["r"], d["dy"], d["rate"], d["i"], d["state"], d["dso"])
    for _ in range(3):
        again = ttt.ttt_lru_forward(*a, **kw)
        assert all(torch.equal(p, q) for p, q in zip(first, again))
        h = ttt.ttt_lru_backward(d["x"], d["r"], d["dy"], d["rate"], d["i"], d["state"], d["dso"])
        assert all(torch.equal(g[k], h[k]) for k in g)


def test_refusals():
    d = _inputs(2, 10, 16, BF, 11)
    x, r = d["x"], d["r"]
    with pytest.raises(TypeError):
        ttt.ttt_lru_forward(x.half(), r)
    with pytest.raises(TypeError):
        ttt.ttt_lru_forward(x, r.float())
    with pytest.raises(ValueError):
        ttt.ttt_lru_forward(x, r[:, :9])
    with pytest.raises(ValueError):
        ttt.ttt_lru_forward(x.cpu(), r)
    with pytest.raises(ValueError):
        ttt.ttt_lru_forward(x.transpose(1, 2), r.transpose(1, 2))
    with pytest.raises(TypeError):
        ttt.ttt_lru_forward(x, r, rate=d["rate"].bfloat16())
    with pytest.raises(ttt.TTTError):
        ttt.ttt_lru_forward(x, r, y=x)
    with pytest.raises(ttt.TTTError):
        ttt.ttt_lru_forward(torch.zeros(2, 300, 16, device="cuda"), torch.zeros(2, 300, 16, device="cuda"),
                            workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ttt.ttt_lru_backward(x, r, d["dy"], grads={"dx": torch.empty_like(x)})
    with pytest.raises(ttt.TTTError):  # y over the state
        over = d["state"].view(BF).flatten()[:32].view(2, 16)
        ttt.ttt_lru_step(x[:, 0], r[:, 0], d["state"], y=over)
