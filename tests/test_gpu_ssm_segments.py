"""The state space scan where a workgroup walks several 64-token chunks, and
where a lane of the vector walk holds two or four values, against 64 bits.

How a sequence is cut goes by the number of heads: with B H >= 192 the
backward on the matrix cores takes segments of up to four chunks and the
forward of two or three, with B H >= 768 (512 for N > 64) the forward walks
the whole sequence. The vector walk takes two values a lane for up to 32
features and four for more where B H ceil(L / 64) >= 512.

Bounds (block_ref.check). A term passes at most L decays, each a few half steps
of fp32: 4 L + 128 of them at the sum of the terms' magnitudes. On the matrix
cores a term of y takes at most two operands rounded to bf16 (the state's
weighted rows and its copy, or the decayed products), one of dx one (the
decayed products, or the state's gradient), dB and dC none that two parts do
not hold: two half steps of bf16 at the same sum. The decay's gradient is a
difference of sums that decay_sums gives, each term as above in fp32.
"""
import pytest
import torch

from tests import block_ref as R
from tests import scan_ref as S
from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _inputs(case, seed, positive=False):
    B, L, H, P, G, N, dt, lens, kind = case
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    speed = {"slow": -4.0, "fast": 1.0, "reset": -2.0, "grow": -5.0}[kind]
    A = torch.exp(r(H).clamp(-1.5, 1.5) + speed)
    z = r(B, L, H)
    if kind == "reset":  # in some chunks the state is forgotten, in others not
        z[:, 70:120:7] = 120.0
        z[:, 200::64] = 120.0
    d = {"x": r(B, L, H, P).to(dt), "dt": z.to(dt), "A": A if kind == "grow" else -A,
         "Bm": (N ** -0.5 * r(B, L, G, N)).to(dt), "Cm": r(B, L, G, N).to(dt), "D": 1 + 0.3 * r(H),
         "dt_bias": r(H) - 3, "state": r(B, H, N, P)}
    dy, dso = r(B, L, H, P).to(dt), r(B, H, N, P)
    if positive:
        d.update({k: d[k].abs() for k in ("x", "Bm", "Cm", "D", "state")})
        dy, dso = dy.abs(), dso.abs()
    d = {k: t.cuda() for k, t in d.items()}
    return d, dy.cuda(), dso.cuda(), None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()


def _poison(d, dy, n):
    if n is not None:
        for b, k in enumerate(n.tolist()):
            for t in (d["x"], d["dt"], d["Bm"], d["Cm"], dy):
                t[b, k:] = float("nan")


def _check(got, ref, name, ops, mag, roundings=0.0):
    R.check(got, ref.cpu(), name, ops, mag.cpu(), roundings)


def _args(d):
    return [d[k] for k in ("x", "dt", "A", "Bm", "Cm")]


CHUNKS = [  # B, L, H, P, G, N, dtype, lens, decay
    (2, 450, 96, 64, 2, 64, BF, [450, 300], "slow"),
    (4, 520, 48, 16, 4, 16, BF, [520, 70, 200, 0], "reset"),
    (1, 256, 192, 64, 1, 128, BF, None, "reset"),
    (2, 300, 96, 33, 1, 20, BF, [300, 129], "slow"),
    (4, 260, 48, 64, 1, 32, BF, None, "fast"),
    (2, 330, 96, 40, 2, 72, BF, [193, 330], "grow"),
    (2, 256, 96, 64, 1, 50, BF, [256, 255], "slow"),
    (2, 256, 96, 24, 1, 40, BF, None, "reset"),
    (2, 256, 96, 64, 1, 64, BF, [65, 192], "grow"),
]
WHOLE = [  # the forward's sequence in one segment
    (16, 200, 48, 16, 1, 16, BF, [200, 65, 0, 128] * 4, "slow"),
    (8, 200, 96, 64, 1, 64, BF, None, "reset"),
    (8, 140, 64, 64, 2, 128, BF, [140] * 7 + [66], "slow"),
]
LANES = [  # the vector walk
    (16, 70, 16, 24, 4, 40, F32, [70, 1, 0, 65] * 4, "slow"),
    (16, 70, 16, 48, 2, 24, F32, None, "fast"),
    (16, 70, 16, 100, 1, 20, BF, [70, 33] * 8, "reset"),
    (16, 130, 16, 64, 1, 64, F32, None, "grow"),
]


@pytest.mark.parametrize("case", CHUNKS + WHOLE + LANES, ids=str)
def test_forward(case):
    d, dy, _, n = _inputs(case, 1)
    ref = {k: S.t64(v) for k, v in d.items()}
    want, mag = S.scan(ref, n), S.scan(S.absolute(ref), n)
    _poison(d, dy, n)
    y, so = ttt.ttt_ssm_forward(*_args(d), d["D"], d["dt_bias"], d["state"], n)
    ops = 4 * case[1] + 128
    _check(y, want["y"], "y", ops, mag["y"], 2.0 if case[6] is BF and case[3] <= 64 else 0.0)
    _check(so, want["state_out"], "state_out", ops, mag["state_out"])


@pytest.mark.parametrize("positive", [False, True], ids=["signed", "positive"])
@pytest.mark.parametrize("case", CHUNKS + LANES, ids=str)
def test_backward(case, positive):
    """Positive operands: no sum cancels, so that the bounds of the decay's
    gradient are close to it."""
    d, dy, dso, n = _inputs(case, 2, positive)
    ref, rdy, rso = {k: S.t64(v) for k, v in d.items()}, S.t64(dy), S.t64(dso)
    want = S.scan(ref, n, rdy, rso)
    mag = S.scan(S.absolute(ref), n, rdy.abs(), rso.abs())
    _poison(d, dy, n)
    got = ttt.ttt_ssm_backward(*_args(d), dy, d["D"], d["dt_bias"], d["state"], dso, n)
    ops, rounded = 4 * case[1] + 128, 2.0 if case[6] is BF and case[3] <= 64 else 0.0
    for k in ("dx", "dB", "dC"):
        _check(got[k], want[k], k, ops, mag[k], rounded)
    _check(got["dstate"], want["dstate"], "dstate", ops, mag["dstate"])
    _check(got["dD"], want["dD"], "dD", ops, mag["dD"])
    q = S.decay_sums(mag, ops)
    mdt = (q * ref["A"].abs() + mag["xdu"]) * mag["sig"]
    _check(got["ddt"], want["ddt"], "ddt", ops, mdt)
    _check(got["dA"], want["dA"], "dA", ops, (q * mag["step"]).sum((0, 1)))
    _check(got["ddt_bias"], want["ddt_bias"], "ddt_bias", ops, mdt.sum((0, 1)))


@pytest.mark.parametrize("case", [CHUNKS[0], CHUNKS[1], CHUNKS[2], LANES[1]], ids=str)
def test_repeats_bit_for_bit(case):
    """Segments of several chunks, forwards and backwards, the same bits each time."""
    d, dy, dso, n = _inputs(case, 3)
    first = None
    for _ in range(6):
        y, so = ttt.ttt_ssm_forward(*_args(d), d["D"], d["dt_bias"], d["state"], n)
        got = ttt.ttt_ssm_backward(*_args(d), dy, d["D"], d["dt_bias"], d["state"], dso, n)
        got.update(y=y, state_out=so)
        if first is None:
            first = {k: t.clone() for k, t in got.items()}
        for k, t in got.items():
            assert torch.equal(t, first[k]), k
            t.fill_(float("nan"))  # what the allocator hands out next
