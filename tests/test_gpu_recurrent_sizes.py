"""The gated linear recurrence and the 8-bit products at the ends of the sizes and
layouts that their header grants."""
import pytest
import torch

from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


@pytest.mark.parametrize("row,at", [(5003, 1), (5008, 1), (5008, 2), (4001, 0)])
def test_a_workspace_as_large_as_the_query_says(row, at):
    """Rows with a dimension of one between them, which is not the rows' stride."""
    g = torch.Generator().manual_seed(1)
    buf = torch.randint(-128, 128, (100, row), generator=g).to(I8).cuda()
    x = buf[:, :3968].unflatten(1, (4, 992))[:, at:at + 1]
    w = torch.randint(-128, 128, (40, 992), generator=g).to(I8).cuda()
    xs, ws = torch.rand(100, 1, generator=g).cuda() + 0.1, torch.rand(40, generator=g).cuda() + 0.1
    n = ttt.ttt_i8_project_workspace(100, x, w)
    y = ttt.ttt_i8_project(x, xs, w, ws, dtype=F32, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
    assert y.shape == (100, 1, 40)
    assert torch.equal(y[:, 0], ttt.ttt_i8_project(x[:, 0].contiguous(), xs[:, 0], w, ws, dtype=F32))
