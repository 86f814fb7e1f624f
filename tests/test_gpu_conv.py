"""The short causal convolution on the GPU against its definition in 64 bits:
each tap count and type, lengths of zero and one, ragged batches, strided
slices, single tokens after a prompt, and its gradients.

Bounds (block_ref.check): a row is K products and sums and an activation of a
few fp32 operations, each off by half a step of fp32 at most, at magnitudes up
to sum |w||x| + |b|; the hardware exp and reciprocal are off by a few steps:
32 half steps hold them all. A weight gradient sums n terms along a chain of at
most n / 16 + 64 additions: that many half steps at the sum of |terms|.
"""
import pytest
import torch

from tests import block_ref as R
from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _inputs(B, L, C, K, dt, seed=0, bias=True, state=True, lens=None, wide=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    d = {"x": r(B, L, C + wide).to(dt).cuda()[..., wide:], "w": (r(C, K) * K ** -0.5).cuda(),
         "bias": (0.3 * r(C)).cuda() if bias else None,
         "state": r(B, K - 1, C).to(dt).cuda() if state else None,
         "dy": r(B, L, C).to(dt).cuda(), "dso": r(B, K - 1, C).to(dt).cuda(),
         "lens": None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda()}
    return d


def _poison(d):
    """NaN in every padded row: it must not be read."""
    if d["lens"] is not None:
        for b, n in enumerate(d["lens"].tolist()):
            d["x"][b, n:] = float("nan")
            d["dy"][b, n:] = float("nan")
    return d


CASES = [  # B, L, C, K, dtype, act, bias, state, lens, wide
    (2, 37, 64, 4, BF, "silu", True, True, None, 8),
    (1, 1, 8, 4, BF, "silu", True, False, None, 0),
    (3, 2, 24, 3, F32, "silu", False, True, None, 4),
    (2, 19, 7, 2, F32, "none", True, True, None, 1),
    (4, 130, 40, 4, BF, "silu", True, True, [0, 1, 130, 77], 3),
    (3, 65, 33, 3, BF, "none", True, False, [65, 2, 0], 0),
    (2, 300, 2176, 4, BF, "silu", True, True, None, 0),
    (2, 257, 771, 3, F32, "silu", True, True, [257, 100], 0),
    (2, 0, 16, 4, BF, "silu", True, True, None, 0),
]


def _ref(d, act):
    x, w, b, s = (R.t64(d[k]) for k in ("x", "w", "bias", "state"))
    n, keep = R.live(d["lens"], x.shape[0], x.shape[1])
    x = torch.where(keep[..., None], x, 0.0)
    return x, w, b, s, R.conv(x, w, b, s, act, d["lens"])


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    B, L, C, K, dt, act, bias, state, lens, wide = case
    d = _poison(_inputs(B, L, C, K, dt, 1, bias, state, lens, wide))
    x, w, b, s, (y, so) = _ref(d, act)
    got, gso = ttt.ttt_conv_forward(d["x"], d["w"], d["bias"], d["state"], act, d["lens"])
    mag = R.conv(x.abs(), w.abs(), None if b is None else b.abs(), None if s is None else s.abs(), "none",
                 d["lens"])[0]
    R.check(got, y, "y", 32, mag)
    assert torch.equal(gso.cpu().to(R.F64), so)
    # the state may be replaced where it stands
    if state:
        st = d["state"].clone()
        got2, st2 = ttt.ttt_conv_forward(d["x"], d["w"], d["bias"], st, act, d["lens"], state_out=st)
        assert st2.data_ptr() == st.data_ptr() and torch.equal(st, gso) and torch.equal(got2, got)


@pytest.mark.parametrize("dt,K,C,wide", [(BF, 4, 64, 0), (F32, 3, 33, 5), (BF, 2, 17, 3), (BF, 4, 2176, 8)])
def test_single_tokens_continue_a_prompt(dt, K, C, wide):
    """Steps after a prompt give the bits of one prompt over all tokens."""
    B, L, T = 3, 9, 6
    d = _inputs(B, L + T, C, K, dt, 2, wide=wide)
    whole, wso = ttt.ttt_conv_forward(d["x"], d["w"], d["bias"], d["state"])
    _, st = ttt.ttt_conv_forward(d["x"][:, :L], d["w"], d["bias"], d["state"])
    for t in range(L, L + T):
        y = ttt.ttt_conv_step(d["x"][:, t], d["w"], st, d["bias"])
        assert torch.equal(y, whole[:, t]), t
    assert torch.equal(st, wso)


def _spread(m):
    return m + m.max() if m.numel() else m


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    B, L, C, K, dt, act, bias, state, lens, wide = case
    d = _poison(_inputs(B, L, C, K, dt, 3, bias, state, lens, wide))
    x, w, b, s, _ = _ref(d, act)
    _, keep = R.live(d["lens"], B, L)
    dy = torch.where(keep[..., None], R.t64(d["dy"]), 0.0)
    dso = R.t64(d["dso"])
    ref = R.gradients(lambda x, w, bias, state: R.conv(x, w, bias, state, act, d["lens"]),
                      {"x": x, "w": w, "bias": b, "state": s}, (dy, dso))
    got = ttt.ttt_conv_backward(d["x"], d["w"], d["dy"], d["bias"], d["state"], d["dso"], act, d["lens"])
    # magnitudes: |act'| <= 1.1
    up = R.gradients(lambda x, w, bias, state: R.conv(x, w, bias, state, "none", d["lens"]),
                     {"x": x.abs(), "w": w.abs(), "bias": b, "state": None if s is None else s.abs()},
                     (1.1 * dy.abs(), dso.abs()))
    # act'(z) is off by what z is off by: half steps of sum |w||x|, at most 8 here
    R.check(got["dx"], ref["x"], "dx", 48, _spread(up["x"]))
    chain = B * L / 16 + 64
    R.check(got["dweight"], ref["w"], "dweight", chain + 48, up["w"])
    if bias:
        R.check(got["dbias"], ref["bias"], "dbias", chain + 48, up["bias"])
    if state:
        R.check(got["dstate"], ref["state"], "dstate", 48, _spread(up["state"]))
    assert set(got) == {"dx", "dweight"} | ({"dbias"} if bias else set()) | ({"dstate"} if state else set())


def test_gradients_into_slices_of_one_buffer():
    """dx may be a slice of a wider buffer, whose other columns stay."""
    d = _inputs(2, 21, 24, 4, BF, 4)
    ref = ttt.ttt_conv_backward(d["x"], d["w"], d["dy"], d["bias"], d["state"], d["dso"])
    wide = torch.full((2, 21, 40), 7.0, dtype=BF, device="cuda")
    g = {k: torch.empty_like(v) for k, v in ref.items()}
    g["dx"] = wide[..., 8:32]
    ttt.ttt_conv_backward(d["x"], d["w"], d["dy"], d["bias"], d["state"], d["dso"], grads=g)
    assert torch.equal(g["dx"], ref["dx"]) and torch.equal(g["dweight"], ref["dweight"])
    assert bool((wide[..., :8] == 7).all()) and bool((wide[..., 32:] == 7).all())
