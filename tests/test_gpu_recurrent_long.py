"""The gated linear recurrence against 64 bits where it is long: prompts by the
longest tiles. Bounds: tests/lru_ref.py's."""
import pytest
import torch

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
