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


def _overlapping(M, K, seed):
    """[M,K] in bf16 whose rows are one value apart: M different rows in M + K values."""
    x = torch.randn(M + K, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(BF)
    return x.as_strided((M, K), (1, 1))


def test_as_many_rows_as_the_quantiser_takes():
    """2^24 rows of a workgroup each: 2^32 threads. The same bits as two calls of half as many."""
    M, K = 1 << 24, 257
    x = _overlapping(M, K, 2)
    q, s = ttt.ttt_i8_quantize(x)
    assert bool((s > 0).all())
    for half in (slice(M // 2), slice(M // 2, M)):
        q2, s2 = ttt.ttt_i8_quantize(x[half])
        assert torch.equal(q[half], q2) and torch.equal(s[half], s2)


def test_as_many_tokens_as_a_product_of_features_takes():
    M, K = 1 << 24, 257
    x = _overlapping(M, K, 3)
    w, ws = ttt.ttt_i8_quantize(torch.randn(3, K, generator=torch.Generator().manual_seed(4)).cuda())
    y = ttt.ttt_i8_linear(x, w, ws)
    assert torch.equal(y[:M // 2], ttt.ttt_i8_linear(x[:M // 2], w, ws))
    assert torch.equal(y[M // 2:], ttt.ttt_i8_linear(x[M // 2:], w, ws))


@pytest.mark.parametrize("B,D", [(4099, 1 << 20), (65535, 65600)])
def test_states_of_more_values_than_32_bits_count(B, D):
    """No tokens at all: states of 2^32 values and more pass through, and their gradients."""
    none = torch.empty(B, 0, D, dtype=BF, device="cuda")
    h = torch.empty(B, D, device="cuda")
    for b in range(0, B, 997):
        h[b:b + 997] = torch.arange(b, min(b + 997, B), device="cuda")[:, None] * 0.5 + torch.arange(D, device="cuda") * 2.0 ** -10
    assert h.numel() > 1 << 32
    _, so = ttt.ttt_lru_forward(none, none, state=h)
    assert torch.equal(so, h)
    _, so = ttt.ttt_lru_forward(none, none, state_out=so)
    assert not bool(so.any())
    g = ttt.ttt_lru_backward(none, none, none, state=so, dstate_out=h)
    assert torch.equal(g["dstate"], h)
    g = ttt.ttt_lru_backward(none, none, none, state=h, grads=g)
    assert not bool(g["dstate"].any())


def test_a_token_of_as_many_states():
    """One token of 2^32 values of state beside the same sequences in two calls."""
    B, D = 4100, 1 << 20
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(B + D, generator=g, device="cuda").to(BF).as_strided((B, 1, D), (1, D, 1))
    y, so = ttt.ttt_lru_forward(x, x)
    for part in (slice(0, 2000), slice(2000, B)):
        y2, so2 = ttt.ttt_lru_forward(x[part], x[part])
        assert torch.equal(y[part], y2) and torch.equal(so[part], so2)


def test_gradients_of_a_token_of_as_many_states():
    B, D = 4100, 1 << 20
    g = torch.Generator("cuda").manual_seed(6)
    x, dy = (torch.randn(B + D, generator=g, device="cuda").to(BF).as_strided((B, 1, D), (1, D, 1)) for _ in range(2))
    rate = 0.5 + torch.rand(D, generator=g, device="cuda")
    got, sums = ttt.ttt_lru_backward(x, x, dy, rate), []
    for part in (slice(0, 2000), slice(2000, B)):
        p = ttt.ttt_lru_backward(x[part], x[part], dy[part], rate)
        assert torch.equal(got["dx"][part], p["dx"]) and torch.equal(got["dr"][part], p["dr"])
        sums.append(p["drate"])
    # a token's share is |dy x| sigma(r) a^2 / s, where sigma a^2 / s is below 0.5 for these rates, and |dy x| 2/pi in
    # the mean: 4100 of them come to less than 2050; sums of them in two orders, at most 100 roundings each
    assert float((got["drate"] - sums[0] - sums[1]).abs().max()) <= 2050 * 200 * 2.0 ** -24
