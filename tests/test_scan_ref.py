"""The batched reference of the scan against the plain definition, torch's
differentiation of it and central differences, all in 64 bits on the CPU."""
import pytest
import torch

from tests import block_ref as R
from tests import scan_ref as S

NAMES = {"x": "dx", "dt": "ddt", "A": "dA", "Bm": "dB", "Cm": "dC", "D": "dD", "dt_bias": "ddt_bias", "state": "dstate"}


def _operands(B, L, H, P, G, N, seed, bare=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    v = {"x": r(B, L, H, P), "dt": r(B, L, H), "A": -torch.exp(r(H)), "Bm": r(B, L, G, N), "Cm": r(B, L, G, N),
         "D": r(H), "dt_bias": r(H) - 2, "state": r(B, H, N, P)}
    if bare:
        v.update(D=None, dt_bias=None, state=None)
    return v, r(B, L, H, P), r(B, H, N, P)


@pytest.mark.parametrize("case", [(2, 9, 4, 3, 2, 5, None, False), (3, 70, 2, 2, 1, 3, [70, 0, 66], False),
                                  (1, 5, 2, 4, 1, 2, None, True)], ids=str)
def test_equals_the_definition_and_its_differentiation(case):
    B, L, H, P, G, N, lens, bare = case
    v, dy, dso = _operands(B, L, H, P, G, N, 1, bare)
    n = None if lens is None else torch.tensor(lens)
    got = S.scan(v, n, dy, dso)
    y, so = R.scan(**v, lens=n)
    assert torch.allclose(got["y"], y, rtol=1e-12, atol=1e-12)
    assert torch.allclose(got["state_out"], so, rtol=1e-12, atol=1e-12)
    want = R.gradients(lambda **w: R.scan(**w, lens=n), v, (dy, dso))
    assert {NAMES[k] for k in want} == set(NAMES.values()) & set(got)
    for k, w in want.items():
        assert torch.allclose(got[NAMES[k]], w, rtol=1e-10, atol=1e-10), k


def test_equals_differences():
    v, dy, dso = _operands(2, 7, 2, 3, 1, 4, 2)
    got = S.scan(v, None, dy, dso)
    g = torch.Generator().manual_seed(3)

    def loss(w):
        o = S.scan(w)
        return float((o["y"] * dy).sum() + (o["state_out"] * dso).sum())

    h = 1e-5
    for k, name in NAMES.items():
        way = torch.randn(v[k].shape, generator=g, dtype=torch.float64)
        along = (loss({**v, k: v[k] + h * way}) - loss({**v, k: v[k] - h * way})) / (2 * h)
        have = float((got[name] * way).sum())
        assert abs(have - along) <= 1e-7 * float((got[name] * way).abs().sum() + 1), name


def test_the_sums_that_bound_the_decay_gradient():
    """q_t = q_{t+1} + row_t - col_t, and a chunk's first q is its border's."""
    v, dy, dso = _operands(1, 130, 2, 2, 1, 3, 4)
    o = S.scan(v, None, dy, dso)
    q, step = o["q"], o["row"] - o["col"]
    assert torch.allclose(q[:, :-1], q[:, 1:] + step[:, :-1], rtol=1e-9, atol=1e-9)
    assert torch.equal(o["ends"], q[:, ::64])
