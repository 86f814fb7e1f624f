"""Workspace queries of the operators around the layer refuse sizes that the
ABI's 32-bit integers do not hold."""
import pytest

from test_sequence_layer_ttt_amd import ttt

QUERIES = [(ttt.ttt_conv_backward_workspace, (2, 8, 16, 4)), (ttt.ttt_ssm_forward_workspace, (2, 8, 4, 64, 2, 32)),
           (ttt.ttt_ssm_backward_workspace, (2, 8, 4, 64, 2, 32)), (ttt.ttt_block_norm_backward_workspace, (2, 8, 64, 3))]


@pytest.mark.parametrize("fn,args", QUERIES, ids=lambda v: getattr(v, "__name__", ""))
def test_sizes_past_32_bits(fn, args):
    assert fn(*args) > 0
    for i in range(len(args)):
        with pytest.raises(ValueError, match="too large"):
            fn(*args[:i], args[i] + 2**32, *args[i + 1:])
        with pytest.raises(ttt.TTTError):
            fn(*args[:i], -1, *args[i + 1:])
