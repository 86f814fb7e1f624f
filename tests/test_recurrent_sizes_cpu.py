"""Workspace queries of the 8-bit products in Python: they answer for the rows
that the calls take, whatever dimensions these come in. And the tiles that the
recurrence takes by size, by which its tests choose theirs."""
import ctypes

import pytest
import torch

from tests import lru_tiles as T
from test_sequence_layer_ttt_amd import _lib, ttt

I8 = torch.int8


def _project(M, K, N, x, xs, w, ws):
    """Bytes by the C ABI for rows that are given by address and stride."""
    n = ctypes.c_size_t(0)
    one = lambda v: ctypes.byref(ctypes.c_int64(v))
    assert _lib.load().ttt_i8_project_workspace(M, K, N, x.data_ptr(), one(xs), w.data_ptr(), one(ws), ctypes.byref(n)) == _lib.TTT_OK
    return n.value


def _buffer(rows, row):
    """[rows, row] of bytes from a 16-byte address on."""
    flat = torch.zeros(rows * row + 16, dtype=I8)
    off = -flat.data_ptr() % 16
    return flat[off:off + rows * row].view(rows, row)


VIEWS = {  # x [...,K] over `rows` rows, the stride between these
    "middle of one": (lambda: _buffer(100, 5003)[:, :3968].unflatten(1, (4, 992))[:, 1:2], 5003),
    "whole chunks, middle of one": (lambda: _buffer(100, 5008)[:, :3968].unflatten(1, (4, 992))[:, 1:2], 5008),
    "odd middle of one, whole rows": (lambda: _buffer(100, 4096).as_strided((100, 1, 992), (4096, 7, 1)), 4096),
    "two of one": (lambda: _buffer(100, 1001).as_strided((100, 1, 1, 992), (1001, 16, 32, 1)), 1001),
    "first of one": (lambda: _buffer(100, 1001)[None, :, :992], 1001),
    "two dimensions of rows": (lambda: _buffer(100, 1008).view(20, 5, 1008)[..., :992], 1008),
    "rows that repeat": (lambda: _buffer(1, 992).expand(100, 992), 0),
}


@pytest.mark.parametrize("name", VIEWS)
def test_a_dimension_of_one_has_no_say_in_the_stride(name):
    make, stride = VIEWS[name]
    x, w = make(), _buffer(32, 992)
    assert x.numel() == 100 * 992
    assert ttt.ttt_i8_project_workspace(100, x, w) == _project(100, 992, 32, x, stride, w, 992)


def test_one_row_has_no_stride():
    row = _buffer(3, 1001)[1:2, :992]
    for x in (row, row[0], row[None]):
        assert ttt.ttt_i8_project_workspace(100, x, _buffer(32, 992)) == _project(100, 992, 32, x, 992, _buffer(32, 992), 992)


@pytest.mark.parametrize("case", T.LONG, ids=str)
def test_sizes_of_the_longest_tiles(case):
    B, L, D, dt, _, gate, _ = case
    assert T.forward_tokens(B, L, D, dt, gate) == 128


# B, L, D, type, gate: the tile's tokens by the width of a thread's loads, input gates and columns
TOKENS = [((32, 2040, 136, torch.bfloat16, False), 128), ((32, 2040, 136, torch.bfloat16, True), 64),
          ((15, 4400, 136, torch.bfloat16, True), 128), ((15, 4400, 137, torch.bfloat16, True), 64),
          ((32, 1930, 136, torch.float32, False), 64), ((32, 2040, 137, torch.float32, False), 64),
          ((32, 1900, 136, torch.bfloat16, False), 64), ((32, 900, 136, torch.bfloat16, True), 32),
          ((1, 300, 136, torch.float32, True), 32)]


@pytest.mark.parametrize("sizes,tokens", TOKENS, ids=str)
def test_tiles_by_size(sizes, tokens):
    assert T.forward_tokens(*sizes) == tokens


def test_queries_refuse_a_weight_that_the_calls_refuse():
    """Three projections' weight counts 3 rows by its first dimension."""
    w = torch.zeros(3, 128, 64, dtype=I8)
    for bad in (w, w[0, 0]):
        with pytest.raises(ValueError, match="2 dimensions"):
            ttt.ttt_i8_linear_workspace(100, bad)
        with pytest.raises(ValueError, match="2 dimensions"):
            ttt.ttt_i8_project_workspace(100, w[0], bad)
    assert ttt.ttt_i8_linear_workspace(100, w.flatten(0, 1)) == 100 * 128 + 400
