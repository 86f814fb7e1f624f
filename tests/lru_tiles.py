"""Sizes of the recurrence's tests by the tiles that they run, with the tile's
length as the library itself chooses it."""
from __future__ import annotations

import ctypes

import torch

from test_sequence_layer_ttt_amd import _lib

BF, F32 = torch.bfloat16, torch.float32


def forward_tokens(B, L, D, dt, gate):
    """Tokens of a prompt's tile for contiguous features: a thread takes 16 bytes of
    channels, or one value where D is no multiple of that."""
    fn = _lib.load()._ZN3ttt18lru_forward_tokensEiiiib  # ttt::lru_forward_tokens
    fn.restype, fn.argtypes = ctypes.c_int, [ctypes.c_int] * 4 + [ctypes.c_bool]
    V = 16 // dt.itemsize
    return fn(B, L, D, V if D % V == 0 else 1, gate)


# B, L, D, type, rate, gate, lens: tiles of 128 tokens
LONG = [
    (32, 2040, 136, BF, False, False, False), (32, 1930, 136, BF, False, False, True),
    (15, 4400, 136, BF, False, True, False), (15, 4400, 136, BF, False, True, True),
    (32, 1930, 136, BF, True, False, True), (15, 4400, 136, BF, True, True, True),
    (16, 4096, 256, BF, False, False, False), (16, 4096, 256, BF, True, False, False),
]
