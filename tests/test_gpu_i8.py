"""8-bit integer products on the GPU against their definition: quantised rows
bit for bit, sums exact at every size, stride and address, outputs within their
roundings.

Bounds: the sum is exact; its conversion to fp32, the two scales and the bias
are a rounding each, 4 half steps of fp32 at |sum| scales + |bias|, and y half a
step of its type.
"""
import pytest
import torch

from tests import block_ref as R
from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


def _quantised(x):
    """The definition: the exact quotient by the fp32 scale, rounded half to even."""
    x = x.cpu().float()
    s = x.abs().amax(-1) / 127
    q = torch.round(x.double() / torch.where(s > 0, s, torch.ones_like(s)).double()[..., None]).clamp(-127, 127)
    return torch.where(s[..., None] > 0, q, 0.0).to(I8), s


def _x(shape, dt, seed, far=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if far:
        x = x * (1 + 9 * (torch.rand(shape[-1], generator=g) < 0.05))
    return x.to(dt)


@pytest.mark.parametrize("shape,dt", [((1, 1), BF), ((3, 7), F32), ((5, 64), BF), ((2, 3, 771), F32), ((4, 2048), BF),
                                      ((5000, 96), BF), ((4100, 33), F32), ((2, 10000), F32), ((1, 65536), BF)], ids=str)
def test_quantize(shape, dt):
    x = _x(shape, dt, 1)
    q, s = ttt.ttt_i8_quantize(x.cuda())
    rq, rs = _quantised(x)
    assert q.dtype == I8 and torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)


@pytest.mark.parametrize("dt", [BF, F32])
def test_quantize_on_borders(dt):
    """Quotients that are whole and a half exactly, and their neighbours in x's type."""
    k = torch.arange(-127, 128, dtype=torch.float64)
    rows = []
    for scale in (1.0, 2.0 ** -7, 3.0, 2.0 ** 40):
        at = torch.cat([k, (k[:-1] + k[1:]) / 2]) * scale
        at = at.to(dt)
        bits = at.view(torch.int16 if dt == BF else torch.int32)
        for d in (0, 1, -1):
            row = (bits + d).view(dt).clone()
            row[at == 0] = 0
            row = torch.where(row.abs() > 127 * scale, torch.full_like(row, 127 * scale), row)
            row[0] = 127 * scale
            rows.append(row)
    x = torch.stack(rows)
    q, s = ttt.ttt_i8_quantize(x.cuda())
    rq, rs = _quantised(x)
    assert torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)


def test_quantize_small_large_and_not_finite():
    inf, nan = float("inf"), float("nan")
    tiny = 2.0 ** -149
    x = torch.tensor([[0, 0, 0, 0], [-0.0, 0, 0, 0], [tiny, 0, -tiny, 0], [200 * tiny, 100 * tiny, -99 * tiny, 63 * tiny],
                      [2.0 ** -126, 2.0 ** -130, -2.0 ** -127, 0], [3e38, -1e38, 1e36, 0], [1, inf, 2, 3], [1, nan, 2, 3],
                      [nan, inf, 0, 0], [1, 2, 3, 4]])
    q, s = ttt.ttt_i8_quantize(x.cuda())
    fine = [0, 1, 2, 3, 4, 5, 9]
    rq, rs = _quantised(x[fine])
    assert torch.equal(s.cpu()[fine], rs) and torch.equal(q.cpu()[fine], rq)
    assert bool(torch.isnan(s[6:9]).all()) and int(q[6:9].abs().max()) == 0
    # and a row like these has no number for an output, the others theirs
    w = torch.ones(3, 4, dtype=I8, device="cuda")
    y = ttt.ttt_i8_linear(x.cuda(), w, torch.ones(3, device="cuda"))
    assert bool(torch.isnan(y[6:9]).all()) and bool(torch.isfinite(y[fine]).all())


def _check(y, x, xs, w, ws, bias, name):
    acc = x.cpu().double().flatten(0, -2) @ w.cpu().double().t()
    ref = acc * xs.cpu().double().reshape(-1, 1) * ws.cpu().double()
    mag = ref.abs()
    if bias is not None:
        ref, mag = ref + bias.cpu().double(), mag + bias.cpu().double().abs()
    R.check(y.flatten(0, -2), ref, name, 4, mag)


def _operands(M, K, N, seed, off=0, row=None, bias=False):
    """8-bit operands whose rows are `row` apart from byte `off` of a buffer on."""
    g = torch.Generator().manual_seed(seed)

    def rows(n):
        r = row or K
        buf = torch.randint(-128, 128, (off + n * r + 16,), generator=g).to(I8).cuda()
        return buf[off:off + n * r].view(n, r)[:, :K]

    return (rows(M), torch.rand(M, generator=g).cuda() + 0.1, rows(N), torch.rand(N, generator=g).cuda() + 0.1,
            torch.randn(N, generator=g).cuda() * 100 if bias else None)


SIZES = [  # M, K, N, first byte, row, out type, bias
    (1, 1, 1, 0, None, F32, False), (1, 16, 1, 0, None, BF, True), (2, 3, 5, 1, None, F32, True),
    (1, 2048, 2048, 0, None, BF, False), (7, 771, 33, 0, None, F32, True), (16, 64, 16, 0, None, BF, False),
    (17, 128, 130, 0, 160, F32, False), (33, 130, 64, 2, 131, BF, True), (64, 2048, 192, 0, None, BF, False),
    (65, 256, 255, 0, None, F32, False), (100, 1000, 77, 3, 1003, BF, True), (128, 96, 128, 0, 112, BF, False),
    (257, 384, 300, 0, None, BF, True), (300, 144, 520, 0, None, F32, True), (513, 80, 514, 0, 96, BF, False),
    (1000, 512, 768, 0, None, BF, False), (31, 8192, 48, 0, None, F32, False), (64, 16, 6144, 0, None, BF, False),
    (5, 4096, 1000, 16, 4112, F32, True), (260, 2064, 260, 0, None, BF, False),
]


@pytest.mark.parametrize("case", SIZES, ids=str)
def test_project(case):
    M, K, N, off, row, dt, bias = case
    x, xs, w, ws, b = _operands(M, K, N, 2, off, row, bias)
    y = ttt.ttt_i8_project(x, xs, w, ws, b, dtype=dt)
    assert y.dtype == dt
    _check(y, x, xs, w, ws, b, "y")
    # into columns of a wider buffer, whose others stay
    wide = torch.full((M, N + 7), 7.0, dtype=dt, device="cuda")
    ttt.ttt_i8_project(x, xs, w, ws, b, dtype=dt, y=wide[:, 3:3 + N])
    assert torch.equal(wide[:, 3:3 + N], y) and bool((wide[:, :3] == 7).all()) and bool((wide[:, 3 + N:] == 7).all())


# sizes that go by each tile shape, in whole steps of K and not, with ragged edges
TILES = [(4090, 256, 4090, BF), (4081, 208, 4094, F32), (2040, 128, 6136, BF), (2033, 512, 6136, BF), (1990, 272, 6130, F32), (2033, 400, 6136, BF),
         (3850, 256, 2040, BF), (4080, 80, 2030, BF), (1000, 512, 768, BF), (700, 48, 900, F32)]


@pytest.mark.parametrize("M,K,N,dt", TILES)
def test_project_by_each_tile_shape(M, K, N, dt):
    x, xs, w, ws, b = _operands(M, K, N, 12, bias=True)
    y = ttt.ttt_i8_project(x, xs, w, ws, b, dtype=dt)
    _check(y, x, xs, w, ws, b, "y")
    assert torch.equal(ttt.ttt_i8_project(x, xs, w, ws, b, dtype=dt), y)


def test_project_at_the_ends_of_its_range():
    """The longest contraction of the lowest values: a sum of 2^30."""
    K = 65536
    for M in (1, 70, 300):
        x, w = (torch.full((n, K), -128, dtype=I8, device="cuda") for n in (M, 40))
        x[0] = 127
        one = torch.ones(max(M, 40), device="cuda")
        y = ttt.ttt_i8_project(x, one[:M], w, one[:40], dtype=F32)
        ref = torch.full((M, 40), 2.0 ** 30)
        ref[0] = -127.0 * 128 * K
        assert torch.equal(y.cpu(), ref)


@pytest.mark.parametrize("lead", [(2, 3), (1, 5), (0, 4), (4, 0), (3, 1, 2)], ids=str)
def test_leading_dimensions(lead):
    x, _, w, ws, b = _operands(1, 48, 21, 3, bias=True)
    x = torch.randint(-128, 128, lead + (48,)).to(I8).cuda()
    xs = torch.rand(lead, device="cuda")
    y = ttt.ttt_i8_project(x, xs, w, ws, b, dtype=F32)
    assert y.shape == lead + (21,)
    _check(y, x, xs, w, ws, b, "y")


@pytest.mark.parametrize("M,K,N,dt,bias", [(1, 2048, 2048, BF, False), (1, 1, 1, F32, True), (3, 100, 40, F32, True),
                                           (8, 768, 96, BF, False), (16, 4096, 64, BF, True), (17, 777, 130, BF, False),
                                           (64, 512, 256, F32, False), (300, 1030, 257, BF, True), (2, 8192, 50, BF, False),
                                           (5, 65536, 3, F32, False), (1100, 128, 512, BF, False)])
def test_linear(M, K, N, dt, bias):
    """From features: the product of the values that the quantiser gives."""
    x = _x((M, K), dt, 4).cuda()
    w, ws = ttt.ttt_i8_quantize(_x((N, K), F32, 5).cuda())
    b = torch.randn(N, generator=torch.Generator().manual_seed(6)).cuda() if bias else None
    y = ttt.ttt_i8_linear(x, w, ws, b)
    q, s = _quantised(x)
    assert y.dtype == dt
    _check(y, q, s, w, ws, b, "y")
    # a strided slice gives the same
    wide = torch.randn(M, K + 24, device="cuda").to(dt)
    wide[:, 8:8 + K] = x
    assert torch.equal(ttt.ttt_i8_linear(wide[:, 8:8 + K], w, ws, b), y)


@pytest.mark.parametrize("B,L,dm,H", [(1, 1, 64, 1), (2, 37, 128, 3), (4, 100, 768, 2), (1, 300, 192, 12), (3, 5, 2048, 4),
                                      (2, 16, 80, 1), (2, 9, 33, 2), (0, 4, 64, 1), (2, 0, 64, 1)])
def test_qkv(B, L, dm, H):
    x = _x((B, L, dm), BF, 7).cuda()
    th, ts = ttt.ttt_i8_quantize(_x((3, H * 64, dm), F32, 8).cuda())
    out = ttt.ttt_qkv_project_i8(x, th, ts, H)
    q, s = _quantised(x) if x.numel() else (x.cpu().to(I8), torch.zeros(B, L))
    for k in range(3):
        assert out[k].shape == (B, H, L, 64)
        _check(out[k].transpose(1, 2).reshape(B, L, H * 64), q, s, th[k], ts[k], None, f"view {k}")


def test_the_same_bits_every_time():
    x, xs, w, ws, b = _operands(100, 2048, 300, 9)
    y = ttt.ttt_i8_project(x, xs, w, ws, dtype=F32)
    f = _x((16, 2048), BF, 10).cuda()
    z = ttt.ttt_i8_linear(f, w, ws)
    for _ in range(3):
        assert torch.equal(ttt.ttt_i8_project(x, xs, w, ws, dtype=F32), y)
        assert torch.equal(ttt.ttt_i8_linear(f, w, ws), z)


def test_refusals():
    x, xs, w, ws, b = _operands(4, 32, 8, 11, bias=True)
    f = x.to(BF)
    for bad in (lambda: ttt.ttt_i8_project(f, xs, w, ws), lambda: ttt.ttt_i8_project(x, xs.double(), w, ws),
                lambda: ttt.ttt_i8_linear(x, w, ws), lambda: ttt.ttt_i8_project(x, xs, w.to(torch.uint8), ws),
                lambda: ttt.ttt_i8_project(x, xs, w, ws, dtype=torch.float16), lambda: ttt.ttt_i8_quantize(x),
                lambda: ttt.ttt_qkv_project_i8(f.float()[None], w[None].expand(3, 8, 32), ws[None].expand(3, 8), 1)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ttt.ttt_i8_project(x, xs[:3], w, ws), lambda: ttt.ttt_i8_project(x, xs, w[:, :31], ws),
                lambda: ttt.ttt_i8_project(x, xs, w, ws[:7]), lambda: ttt.ttt_i8_project(x, xs, w, ws, b[:7]),
                lambda: ttt.ttt_i8_project(x.t(), xs, w, ws), lambda: ttt.ttt_i8_project(x.cpu(), xs, w, ws),
                lambda: ttt.ttt_i8_linear(f.view(2, 2, 32).transpose(0, 1), w, ws),
                lambda: ttt.ttt_qkv_project_i8(f[None], w, ws, 1), lambda: ttt.ttt_qkv_project_i8(f[None], w, ws, -1)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ttt.TTTError):
        ttt.ttt_i8_linear(f, w, ws, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ttt.TTTError):
        ttt.ttt_i8_linear(f, w, ws, workspace=torch.empty(4096, dtype=torch.uint8, device="cuda")[1:])
    with pytest.raises(ttt.TTTError):
        ttt.ttt_i8_quantize(torch.zeros(1, 65537, device="cuda"))
    ox, oxs, ow, ows, _ = _operands(70, 33, 8, 12)
    assert ttt.ttt_i8_project_workspace(70, ox, ow) == 78 * 128
    with pytest.raises(ttt.TTTError):
        ttt.ttt_i8_project(ox, oxs, ow, ows, workspace=torch.empty(78 * 128 - 16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ttt.TTTError):
        ttt.ttt_i8_linear(f, w, ws, y=f[:, :8])
