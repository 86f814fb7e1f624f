"""The selective state space scan on the GPU against its definition in 64 bits,
token by token: both storage types, odd head and state sizes, groups, lengths
of zero and one, ragged batches whose padding holds NaN, strided views, several
segments, single tokens after a prompt, and all gradients.

Bounds (block_ref.check). A state's term passes at most L decays, each a few
half steps of fp32 (expf, softplus, the product): 4 L + 128 half steps at the
sum of the terms' magnitudes hold them, which the same scan of absolute values
gives. Where matrix products take a bf16 operand (the decayed C . B products,
the state, and their counterparts in the gradients), each is off by half a
step of bf16: two of them at that sum. ddt and dA come from running sums over
at most 256 tokens of products dy . y and are bounded by those sums.
"""
import pytest
import torch

from tests import block_ref as R
from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _inputs(B, L, H, P, G, N, dt, seed, lens=None, state=True, D=True, bias=True, slow=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    d = {"x": r(B, L, H, P).to(dt).cuda(), "dt": r(B, L, H).to(dt).cuda(),
         "A": -torch.exp(2.7 * torch.rand(H, generator=g) - (4 if slow else 0)).cuda(),
         "Bm": (N ** -0.5 * r(B, L, G, N)).to(dt).cuda(), "Cm": r(B, L, G, N).to(dt).cuda(),
         "D": (1 + 0.3 * r(H)).cuda() if D else None,
         "dt_bias": (r(H) - 3).cuda() if bias else None,
         "state": r(B, H, N, P).cuda() if state else None}
    dy, dso = r(B, L, H, P).to(dt).cuda(), r(B, H, N, P).cuda()
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()
    return d, dy, dso, n


def _poison(d, dy, n):
    if n is not None:
        for b, k in enumerate(n.tolist()):
            for t in (d["x"], d["dt"], d["Bm"], d["Cm"], dy):
                t[b, k:] = float("nan")


CASES = [  # B, L, H, P, G, N, dtype, lens, state, D, bias, slow decay
    (2, 70, 2, 64, 1, 64, BF, None, True, True, True, False),
    (1, 1, 2, 64, 1, 64, BF, None, True, True, True, False),
    (2, 0, 2, 64, 2, 32, BF, None, True, True, True, False),
    (3, 200, 4, 64, 2, 128, BF, [200, 0, 131], True, True, True, True),
    (1, 330, 2, 64, 1, 64, BF, None, False, False, False, True),
    (2, 129, 3, 64, 1, 32, BF, [1, 129], False, True, True, False),
    (1, 64, 1, 64, 1, 64, BF, None, False, True, True, False),
    (2, 65, 4, 48, 2, 24, F32, [65, 64], True, True, True, False),
    (1, 300, 2, 64, 1, 16, F32, None, True, True, True, True),
    (2, 33, 3, 1, 3, 1, F32, None, True, True, False, False),
    (1, 20, 2, 128, 1, 100, F32, None, False, False, True, False),
    (2, 17, 2, 7, 1, 128, BF, [0, 9], True, True, True, False),
    (2, 150, 4, 16, 2, 16, BF, [150, 3], True, True, True, False),
    (1, 260, 2, 33, 1, 77, BF, None, True, True, True, True),
    (2, 70, 2, 64, 1, 20, BF, None, True, False, True, False),
    (1, 90, 2, 100, 1, 40, BF, None, True, True, True, False),
]


def _absolute(d):
    f = lambda k: None if d[k] is None else d[k].abs()
    return dict(d, x=f("x"), Bm=f("Bm"), Cm=f("Cm"), D=f("D"), state=f("state"))


def _call(fn, d, *a, **kw):
    return fn(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], *a, D=d["D"], dt_bias=d["dt_bias"], **kw)


def _roundings(case):
    return 2.0 if case[6] is BF and case[3] <= 64 else 0.0


def _setup(case, seed):
    B, L, H, P, G, N, dt, lens, state, D, bias, slow = case
    d, dy, dso, n = _inputs(B, L, H, P, G, N, dt, seed, lens, state, D, bias, slow)
    ref, rdy = {k: R.t64(v) for k, v in d.items()}, R.t64(dy)
    _, keep = R.live(n, B, L)
    rdy = torch.where(keep[..., None, None], rdy, 0.0)
    _poison(d, dy, n)
    return d, dy, dso, n, ref, rdy


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    d, _, _, n, ref, _ = _setup(case, 1)
    y, so = R.scan(**ref, lens=n)
    my, ms = R.scan(**_absolute(ref), lens=n)
    ops = 4 * case[1] + 128
    gy, gs = _call(ttt.ttt_ssm_forward, d, state=d["state"], lens=n)
    R.check(gy, y, "y", ops, my, _roundings(case))
    R.check(gs, so, "state_out", ops, ms)
    if d["state"] is not None:  # replaced where it stands
        st = d["state"].clone()
        y2, s2 = _call(ttt.ttt_ssm_forward, d, state=st, state_out=st, lens=n)
        assert s2.data_ptr() == st.data_ptr() and torch.equal(st, gs) and torch.equal(y2, gy)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    d, dy, dso, n, ref, rdy = _setup(case, 2)
    B, L = case[0], case[1]
    rso = R.t64(dso)
    fn = lambda **v: R.scan(**v, lens=n)
    want = R.gradients(fn, ref, (rdy, rso))
    up = _absolute(ref)
    mag = R.gradients(fn, dict(up, dt_in=up["dt"]), (rdy.abs(), rso.abs()))
    got = _call(ttt.ttt_ssm_backward, d, dy, state=d["state"], dstate_out=dso, lens=n)
    names = {"x": "dx", "dt": "ddt", "A": "dA", "Bm": "dB", "Cm": "dC", "D": "dD", "dt_bias": "ddt_bias",
             "state": "dstate"}
    assert set(got) == {names[k] for k in want}
    ops = 4 * L + 128
    for k in ("x", "Bm", "Cm"):
        R.check(got[names[k]], want[k], names[k], ops, mag[k], _roundings(case))
    if "state" in want:
        R.check(got["dstate"], want["state"], "dstate", ops, mag["state"])
    if "D" in want:
        R.check(got["dD"], want["D"], "dD", L + 128, mag["D"] if L else None)
    # q_t: a running sum over up to 256 tokens of dy . y and u . du, and the
    # state's product with its gradient at the segment's end
    my, ms = R.scan(**up, lens=n)
    if not L:
        return
    A = ref["A"].abs()
    rows = (rdy.abs() * my).sum(-1)  # [B,L,H]
    end = (ms * rso.abs()).sum((-1, -2)) if L else 0.0
    window = torch.stack([rows[:, t:t + 256].sum(1) for t in range(L)], 1)
    q = 2 * window + rows.amax(1, keepdim=True) * 4 + end[:, None]
    z = ref["dt"] + (0 if ref["dt_bias"] is None else ref["dt_bias"])
    z = torch.where(R.live(n, B, L)[1][..., None], z, torch.full_like(z, -1e3))
    step, sig = torch.logaddexp(z, torch.zeros_like(z)), 1 / (1 + torch.exp(-z))
    mdt = A * q * sig + mag["dt_in"].abs()
    R.check(got["ddt"], want["dt"], "ddt", ops, mdt)
    R.check(got["dA"], want["A"], "dA", ops, (q * step).sum((0, 1)))
    if "dt_bias" in want:
        R.check(got["ddt_bias"], want["dt_bias"], "ddt_bias", ops, mdt.sum((0, 1)))


@pytest.mark.parametrize("shape", [(2, 2, 64, 1, 64, BF), (3, 4, 48, 2, 24, F32), (1, 1, 7, 1, 5, BF)], ids=str)
def test_single_tokens_continue_a_prompt(shape):
    B, H, P, G, N, dt = shape
    L, T = 37, 5
    d, _, _, _ = _inputs(B, L + T, H, P, G, N, dt, 3)
    ref = {k: R.t64(v) for k, v in d.items()}
    y, so = R.scan(**ref, lens=None)
    my, ms = R.scan(**_absolute(ref), lens=None)
    head = {k: v[:, :L] if k in ("x", "dt", "Bm", "Cm") else v for k, v in d.items()}
    _, st = _call(ttt.ttt_ssm_forward, head, state=d["state"])
    ops = 4 * (L + T) + 128
    for t in range(L, L + T):
        one = {k: v[:, t] if k in ("x", "dt", "Bm", "Cm") else v for k, v in d.items()}
        got = ttt.ttt_ssm_step(one["x"], one["dt"], d["A"], one["Bm"], one["Cm"], st, d["D"], d["dt_bias"])
        R.check(got, y[:, t], f"y[{t}]", ops, my[:, t])
    R.check(st, so, "state", ops, ms)


@pytest.mark.parametrize("dt,P,N", [(BF, 64, 64), (F32, 20, 12)])
def test_views_of_wider_rows_and_of_heads_first_features(dt, P, N):
    """x, B and C as slices of one buffer, then x and y as [B,H,L,P] features,
    give the bits of the contiguous operands; so do slices for the gradients,
    whose neighbours stay."""
    B, L, H, G = 2, 70, 3, 1
    d, dy, dso, _ = _inputs(B, L, H, P, G, N, dt, 4)
    ref, rs = _call(ttt.ttt_ssm_forward, d, state=d["state"])
    row = torch.zeros(B, L, H * P + 2 * N + 8, device="cuda", dtype=dt)
    cut = lambda t: {"x": t[..., 8:8 + H * P].unflatten(-1, (H, P)),
                     "Bm": t[..., 8 + H * P:8 + H * P + N].unflatten(-1, (G, N)),
                     "Cm": t[..., 8 + H * P + N:].unflatten(-1, (G, N))}
    v = dict(d, **cut(row))
    for k in ("x", "Bm", "Cm"):
        v[k].copy_(d[k])
    y, s = _call(ttt.ttt_ssm_forward, v, state=d["state"])
    assert torch.equal(y, ref) and torch.equal(s, rs)
    heads = dict(d, x=d["x"].transpose(1, 2).contiguous().transpose(1, 2))
    out = torch.empty(B, H, L, P, device="cuda", dtype=dt).transpose(1, 2)
    y, s = _call(ttt.ttt_ssm_forward, heads, state=d["state"], y=out)
    assert torch.equal(y, ref) and torch.equal(s, rs)
    gr = _call(ttt.ttt_ssm_backward, d, dy, state=d["state"], dstate_out=dso)
    grow = torch.full_like(row, 5.0)
    g2 = {k: torch.empty_like(t) for k, t in gr.items()}
    g2.update({"d" + k[0]: t for k, t in cut(grow).items()})
    _call(ttt.ttt_ssm_backward, v, dy, state=d["state"], dstate_out=dso, grads=g2)
    for k in gr:
        assert torch.equal(g2[k], gr[k]), k
    assert bool((grow[..., :8] == 5).all())


@pytest.mark.parametrize("dt", [BF, F32])
def test_decay_that_forgets_everything_and_one_that_forgets_nothing(dt):
    """dt so large that a_t is 0 (its logarithm below what exp holds), and so
    small that a_t is 1 and nothing is added."""
    B, L, H, P, G, N = 1, 130, 2, 64, 1, 64
    d, _, _, _ = _inputs(B, L, H, P, G, N, dt, 5)
    d["dt"] = torch.full((B, L, H), 200.0, device="cuda").to(dt)
    ref = {k: R.t64(v) for k, v in d.items()}
    y, so = R.scan(**ref, lens=None)
    my, ms = R.scan(**_absolute(ref), lens=None)
    gy, gs = _call(ttt.ttt_ssm_forward, d, state=d["state"])
    R.check(gy, y, "y", 4 * L + 128, my, 2.0)
    R.check(gs, so, "state_out", 4 * L + 128, ms)
    d["dt"] = torch.full((B, L, H), -200.0, device="cuda").to(dt)
    gy, gs = _call(ttt.ttt_ssm_forward, d, state=d["state"])
    assert torch.equal(gs, d["state"])


@pytest.mark.parametrize("dt", [BF, F32])
def test_states_that_grow(dt):
    """A > 0: factors above 1 between tokens of one chunk, of two and of two segments."""
    B, L, H, P, G, N = 1, 200, 2, 64, 1, 64
    d, dy, dso, _ = _inputs(B, L, H, P, G, N, dt, 6)
    d["A"] = torch.tensor([0.3, 1.0], device="cuda")
    ref = {k: R.t64(v) for k, v in d.items()}
    y, so = R.scan(**ref, lens=None)
    my, ms = R.scan(**_absolute(ref), lens=None)
    gy, gs = _call(ttt.ttt_ssm_forward, d, state=d["state"])
    R.check(gy, y, "y", 4 * L + 128, my, 2.0 if dt is BF else 0.0)
    R.check(gs, so, "state_out", 4 * L + 128, ms)
    want = R.gradients(lambda **v: R.scan(**v, lens=None), ref, (R.t64(dy), R.t64(dso)))
    mag = R.gradients(lambda **v: R.scan(**v, lens=None), _absolute(ref), (R.t64(dy).abs(), R.t64(dso).abs()))
    got = _call(ttt.ttt_ssm_backward, d, dy, state=d["state"], dstate_out=dso)
    for k, n in (("x", "dx"), ("Bm", "dB"), ("Cm", "dC")):
        R.check(got[n], want[k], n, 4 * L + 128, mag[k], 2.0 if dt is BF else 0.0)
    R.check(got["dstate"], want["state"], "dstate", 4 * L + 128, mag["state"])
