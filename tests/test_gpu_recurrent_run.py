"""The gated linear recurrence and the 8-bit products as a model runs them: a
block whose projections are held in 8 bits over ragged prompts and then token by
token, the TTT layer on views that were projected in 8 bits, a training step of
the recurrence; on side streams, two calls at once, captured into graphs that
share a workspace and replayed; rows past 4 GiB; and what a call writes into
given tensors."""
import pytest
import torch

import oracle
from tests import block_ref as R
from tests import lru_ref as Q
from tests import parity as P
from tests.test_gpu_i8 import _check, _quantised
from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8
EPS = 1e-6


def _product(y, x, w, ws, name):
    """An 8-bit product of features against its definition on these features."""
    q, s = _quantised(x)
    _check(y, q, s, w, ws, None, name)


def _recurrence(y, so, x, r, rate, i, state, lens):
    """And the recurrence's."""
    e = [R.t64(t) for t in (x, r, rate, i, state)]
    want, wso = Q.forward(*e, lens)
    b = Q.Bounds(*e, lens)
    Q.check(y, want, "y", torch.where(b.keep, b.E[:, 1:], 0.0))
    Q.check(so, wso, "state", b.E[:, -1])


@pytest.mark.parametrize("dt", [BF, F32])
def test_a_block_in_8_bits_over_ragged_prompts_and_then_token_by_token(dt):
    """Norm, 8-bit projection to features and gates, convolution, recurrence, 8-bit
    output projection, norm: each on what the one before it returns, against its
    definition on those values."""
    dm, D, K, B, L, T = 96, 64, 4, 3, 150, 3
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g)
    post, pre, rate = (1 + 0.1 * r(dm)).cuda(), (1 + 0.1 * r(dm)).cuda(), torch.rand(D, generator=g).cuda()
    w_in, s_in = ttt.ttt_i8_quantize((r(3 * D, dm) * dm ** -0.5).cuda())
    w_out, s_out = ttt.ttt_i8_quantize((r(dm, D) * D ** -0.5).cuda())
    cw, cb = (r(D, K) * K ** -0.5).cuda(), (0.1 * r(D)).cuda()
    lens = torch.tensor([150, 1, 77], dtype=torch.int32).cuda()
    resid, y = r(B, L + T, dm).to(dt).cuda(), r(B, L + T, dm).to(dt).cuda()

    _, x = ttt.ttt_block_norm(resid[:, :L], y[:, :L], post, pre, eps=EPS, lens=lens)
    z = ttt.ttt_i8_linear(x, w_in, s_in)
    _product(z, x, w_in, s_in, "z")
    c, cs = ttt.ttt_conv_forward(z[..., :D], cw, cb, lens=lens)
    h, hs = ttt.ttt_lru_forward(c, z[..., D:2 * D], rate, z[..., 2 * D:], lens=lens)
    _recurrence(h, hs, c, z[..., D:2 * D], rate, z[..., 2 * D:], None, lens)
    o = ttt.ttt_i8_linear(h, w_out, s_out)
    _product(o, h, w_out, s_out, "out")
    assert not bool(o[1, 1:].any())  # rows behind a sequence: zeros all the way
    # each sequence goes on from its own state
    state = hs.clone()
    steps = []
    for t in range(L, L + T):
        _, x = ttt.ttt_block_norm(resid[:, t:t + 1], y[:, t:t + 1], post, pre, eps=EPS)
        z = ttt.ttt_i8_linear(x[:, 0], w_in, s_in)
        _product(z, x[:, 0], w_in, s_in, "z")
        c = ttt.ttt_conv_step(z[:, :D], cw, cs, cb)
        before = state.clone()
        h = ttt.ttt_lru_step(c, z[:, D:2 * D], state, rate, z[:, 2 * D:])
        _recurrence(h[:, None], state, c[:, None], z[:, None, D:2 * D], rate, z[:, None, 2 * D:], before, None)
        o = ttt.ttt_i8_linear(h, w_out, s_out)
        _product(o, h, w_out, s_out, "out")
        steps.append((c, z))
    # the tokens as one prompt from that state
    xs = torch.stack([c for c, _ in steps], 1)
    zs = torch.stack([z for _, z in steps], 1)
    _, again = ttt.ttt_lru_forward(xs, zs[..., D:2 * D], rate, zs[..., 2 * D:], hs)
    assert torch.allclose(again, state, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("B,L,H,dm", [(2, 70, 2, 128), (1, 16, 3, 192)])
def test_the_layer_on_views_projected_in_8_bits(B, L, H, dm):
    g = torch.Generator().manual_seed(B)
    r = lambda *s: torch.randn(s, generator=g)
    x = r(B, L, dm).to(BF).cuda()
    theta, ts = ttt.ttt_i8_quantize((r(3, H * 64, dm) * dm ** -0.5).cuda())
    q, k, v = ttt.ttt_qkv_project_i8(x, theta, ts, H)
    for n, t in enumerate((q, k, v)):
        _product(t.transpose(1, 2).reshape(B, L, H * 64), x, theta[n], ts[n], f"view {n}")
    eta = torch.full((B, H, L), 1 / 64, device="cuda")
    W0, b0, gam, bet = (0.02 * r(H, 64, 64)).cuda(), torch.zeros(H, 64).cuda(), torch.ones(H, 64).cuda(), torch.zeros(H, 64).cuda()
    o, W, b = ttt.ttt_linear_forward(q, k, v, eta, W0, b0, gam, bet)
    want = oracle.linear_forward(*(P.to_np(t) for t in (q, k, v, eta, W0, b0, gam, bet)), EPS)
    for got, ref in zip((o, W, b), want):
        assert P.max_rel(P.to_np(got), ref, B * H) < 2e-2
    # beside the bf16 projection of the same weights: off by what 8 bits round, half a step of 1/127 of
    # the largest of a row in each operand, over dm products
    full = ttt.ttt_qkv_project(x, (theta.float() * ts[..., None]).to(BF), H)
    for a, c in zip((q, k, v), full):
        assert float((a.float() - c.float()).norm() / c.float().norm()) < 0.02


def test_a_training_step_of_the_recurrence():
    """Projection (fp32), recurrence, projection: gradients by the recurrence's
    backward into slices of the projection's, against torch's differentiation of
    the chain in 64 bits and along a direction against differences of it."""
    B, L, dm, D = 2, 90, 24, 16
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g)
    x, dout = r(B, L, dm).cuda(), r(B, L, dm).cuda()
    p = {"w_in": (r(dm, 3 * D) * dm ** -0.5).cuda(), "w_out": (r(D, dm) * D ** -0.5).cuda(), "rate": torch.rand(D, generator=g).cuda(),
         "h0": r(B, D).cuda()}
    z = x @ p["w_in"]
    cols = lambda t: (t[..., :D], t[..., D:2 * D], t[..., 2 * D:])
    fx, fr, fi = cols(z)
    h, _ = ttt.ttt_lru_forward(fx, fr, p["rate"], fi, p["h0"])
    dh = dout @ p["w_out"].t()
    dz = torch.empty_like(z)
    gx, gr, gi = cols(dz)
    grads = {"dx": gx, "dr": gr, "di": gi, "drate": torch.empty_like(p["rate"]), "dstate": torch.empty_like(p["h0"])}
    ttt.ttt_lru_backward(fx, fr, dh, p["rate"], fi, p["h0"], grads=grads)
    got = {"x": dz @ p["w_in"].t(), "w_in": x.flatten(0, 1).t() @ dz.flatten(0, 1),
           "w_out": h.flatten(0, 1).t() @ dout.flatten(0, 1), "rate": grads["drate"], "h0": grads["dstate"]}
    leaves = {"x": R.t64(x), **{k: R.t64(v) for k, v in p.items()}}

    def chain(x, w_in, w_out, rate, h0):
        a, b, c = cols(x @ w_in)
        return (Q.forward(a, b, rate, c, h0, None)[0] @ w_out,)

    want = R.gradients(chain, leaves, (R.t64(dout),))
    for k, w in want.items():
        err = float((R.t64(got[k]) - w).abs().max() / w.abs().max())
        print(f"[lru] d{k}: {err:.1e}", flush=True)
        assert err <= 1e-4, k  # some 1000 half steps of fp32 over the chain and its sums of 180 rows
    d = {k: torch.randn(v.shape, generator=g, dtype=R.F64) for k, v in leaves.items()}
    loss = lambda s: float((chain(**{k: v + s * d[k] for k, v in leaves.items()})[0] * R.t64(dout)).sum())
    along = (loss(1e-5) - loss(-1e-5)) / 2e-5
    have = sum(float((R.t64(got[k]) * d[k]).sum()) for k in want)
    assert abs(have - along) <= 1e-4 * sum(float((want[k] * d[k]).abs().sum()) for k in want)


def _ops(dt=BF, B=2, L=400, D=200, seed=0):
    """Each entry point with its operands and outputs made beforehand:
    name -> (fn(stream), outputs, operands that may change)."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).cuda()
    ops = {}
    x, rr, i, rate, h0 = r(B, L, D).to(dt), r(B, L, D).to(dt), r(B, L, D).to(dt), r(D).abs(), r(B, D)
    y, so = torch.empty_like(x), torch.empty_like(h0)
    ws = torch.empty(ttt.ttt_lru_forward_workspace(B, L, D), dtype=torch.uint8, device="cuda")
    ops["lru_forward"] = (lambda s: ttt.ttt_lru_forward(x, rr, rate, i, h0, y=y, state_out=so, workspace=ws, stream=s), [y, so],
                          [x, rr])
    gr = {"dx": torch.empty_like(x), "dr": torch.empty_like(x), "di": torch.empty_like(x), "drate": torch.empty_like(rate),
          "dstate": torch.empty_like(h0)}
    ws2 = torch.empty(ttt.ttt_lru_backward_workspace(B, L, D), dtype=torch.uint8, device="cuda")
    ops["lru_backward"] = (lambda s: ttt.ttt_lru_backward(x, rr, x, rate, i, h0, h0, workspace=ws2, grads=gr, stream=s),
                           list(gr.values()), [x, rr])
    ty, st = torch.empty(B, D, dtype=dt, device="cuda"), torch.zeros_like(h0)
    ops["lru_step"] = (lambda s: ttt.ttt_lru_step(x[:, 0], rr[:, 0], st, rate, i[:, 0], y=ty, stream=s), [ty, st], [x])
    K, N = 208, 130
    f, q, sc = r(B, L, K).to(dt), torch.empty(B, L, K, dtype=I8, device="cuda"), torch.empty(B, L, device="cuda")
    ops["i8_quantize"] = (lambda s: ttt.ttt_i8_quantize(f, q, sc, stream=s), [q, sc], [f])
    w, wsc = ttt.ttt_i8_quantize(r(N, K))
    q2, sc2 = ttt.ttt_i8_quantize(f)
    py = torch.empty(B, L, N, dtype=dt, device="cuda")
    ops["i8_project"] = (lambda s: ttt.ttt_i8_project(q2, sc2, w, wsc, dtype=dt, y=py, stream=s), [py], [sc2])
    ly = torch.empty(B, L, N, dtype=dt, device="cuda")
    ws3 = torch.empty(ttt.ttt_i8_linear_workspace(B * L, w), dtype=torch.uint8, device="cuda")
    ops["i8_linear"] = (lambda s: ttt.ttt_i8_linear(f, w, wsc, y=ly, workspace=ws3, stream=s), [ly], [f])
    # rows that are laid out anew
    wo, wso = ttt.ttt_i8_quantize(r(N, K - 1))
    qo, oy = q2[..., 1:], torch.empty(B, L, N, dtype=dt, device="cuda")
    ws4 = torch.empty(ttt.ttt_i8_project_workspace(B * L, qo, wo), dtype=torch.uint8, device="cuda")
    ops["i8_project_odd"] = (lambda s: ttt.ttt_i8_project(qo, sc2, wo, wso, dtype=dt, y=oy, workspace=ws4, stream=s), [oy], [sc2])
    fy = torch.empty(B, N, dtype=dt, device="cuda")
    ops["i8_linear_few"] = (lambda s: ttt.ttt_i8_linear(f[:, 0], w, wsc, y=fy, workspace=ws3, stream=s), [fy], [f])
    th, ths = ttt.ttt_i8_quantize(r(3, 128, K))
    X = f.to(BF)
    out = tuple(torch.empty(B, 2, L, 64, dtype=BF, device="cuda") for _ in range(3))
    ops["qkv_project_i8"] = (lambda s: ttt.ttt_qkv_project_i8(X, th, ths, 2, out=out, workspace=ws3, stream=s), list(out), [X])
    return ops


NAMES = ["lru_forward", "lru_backward", "lru_step", "i8_quantize", "i8_project", "i8_project_odd", "i8_linear",
         "i8_linear_few", "qkv_project_i8"]


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", NAMES)
def test_repeats_bit_for_bit_and_on_a_side_stream(name, dt):
    fn, outs, _ = _ops(dt)[name]

    def run(stream):
        for o in outs:
            o.zero_() if name == "lru_step" else o.fill_(3)
        torch.cuda.synchronize()
        fn(stream)
        torch.cuda.synchronize()
        return [o.clone() for o in outs]

    a, b, c = run(None), run(None), run(torch.cuda.Stream())
    for u, v, w in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, w)


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name):
    """Two graphs over one workspace: their replays, with new operands and eager work
    between them, give the eager call's bits each time."""
    fn, outs, ins = _ops(BF)[name]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fn(None)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:
        with torch.cuda.graph(graph):
            fn(None)
    for rep in range(4):
        for t in ins:
            t.copy_(torch.roll(t, 1, 0) * 0.75 + 0.25)
        for o in outs:
            o.zero_()
        fn(None)
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_() if name == "lru_step" else o.fill_(7)
        torch.cuda.synchronize()
        graphs[rep % 2].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), rep
        torch.randn(1 << 16, device="cuda").sum().item()  # eager work of the program's own


@pytest.mark.parametrize("name", ["lru_forward", "lru_backward", "i8_project", "i8_project_odd", "i8_linear"])
def test_two_calls_at_once(name):
    """Two streams, each with its own workspace and outputs."""
    a, b = _ops(BF, L=3000, D=520, seed=1)[name], _ops(BF, L=3000, D=520, seed=2)[name]
    want = []
    for fn, outs, _ in (a, b):
        fn(None)
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
        for o in outs:
            o.fill_(1)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a[0](s1)
        b[0](s2)
    torch.cuda.synchronize()
    for (_, outs, _), w in zip((a, b), want):
        for o, v in zip(outs, w):
            assert torch.equal(o, v)


def test_a_long_prompt_of_many_columns_at_once():
    """More tiles than the chip holds at a time, columns of many sequences: equal to the
    sequences one by one (a sequence's sums do not depend on the others')."""
    B, L, D = 24, 2000, 640
    d = [torch.randn(B, L, D, device="cuda", generator=torch.Generator("cuda").manual_seed(k)).to(BF) for k in range(3)]
    rate = torch.rand(D, device="cuda")
    y, so = ttt.ttt_lru_forward(d[0], d[1], rate, d[2])
    e = [R.t64(t[5:6, :, 600:]) for t in d]
    want, wso = Q.forward(e[0], e[1], R.t64(rate[600:]), e[2], None, None)
    b = Q.Bounds(e[0], e[1], R.t64(rate[600:]), e[2], None, None)
    Q.check(y[5:6, :, 600:], want, "y", b.E[:, 1:])
    Q.check(so[5:6, 600:], wso, "state", b.E[:, -1])
    for _ in range(3):
        again = ttt.ttt_lru_forward(d[0], d[1], rate, d[2])
        assert torch.equal(again[0], y) and torch.equal(again[1], so)


def _normal(*shape):
    x = torch.empty(shape, device="cuda", dtype=BF)
    for part in x.flatten(0, -2).split(1 << 17):
        part.normal_()
    return x


def test_rows_past_4_gib_recurrence():
    """Tokens whose offsets pass 2^31 elements: the tail against a call over its rows
    from the state before them. Twice two roundings to bf16, and some 100 half steps of
    fp32 at the largest value, since the tiles are cut elsewhere."""
    D, L = 2176, (1 << 20) + 37
    x = _normal(1, L, D)
    rate = torch.rand(D, device="cuda") + 0.05
    near = lambda a, b: bool(((a.float() - b.float()).abs() <= 2.0 ** -6 * b.float().abs() + 1e-5 * b.float().abs().max()).all())
    y, so = ttt.ttt_lru_forward(x, x, rate)
    cut = L - 300
    _, st = ttt.ttt_lru_forward(x[:, :cut], x[:, :cut], rate)
    y2, so2 = ttt.ttt_lru_forward(x[:, cut:], x[:, cut:], rate, state=st)
    assert near(y[:, cut:], y2) and near(so, so2)
    g = ttt.ttt_lru_backward(x, x, y, rate)
    g2 = ttt.ttt_lru_backward(x[:, cut:], x[:, cut:], y[:, cut:], rate, state=st)
    assert near(g["dx"][:, cut:], g2["dx"]) and near(g["dr"][:, cut:], g2["dr"])


def test_rows_past_4_gib_products():
    """Operands and outputs whose offsets pass 2^32 bytes: the same bits as short calls."""
    K, M = 65536, (1 << 16) + 200
    x = torch.randint(-128, 128, (M, K), dtype=I8, device="cuda")
    xs = torch.rand(M, device="cuda")
    cut = M - 150
    w, ws = torch.randint(-128, 128, (70, K), dtype=I8, device="cuda"), torch.rand(70, device="cuda")
    y = ttt.ttt_i8_project(x, xs, w, ws)
    assert torch.equal(y[cut:], ttt.ttt_i8_project(x[cut:], xs[cut:], w, ws))
    for m in (3, 70):  # as the weight, few tokens and more
        y = ttt.ttt_i8_project(w[:m], ws[:m], x, xs)
        assert torch.equal(y[:, cut:], ttt.ttt_i8_project(w[:m], ws[:m], x[cut:], xs[cut:]))
    # rows at odd addresses
    o = x.view(-1)[1:].as_strided((M, K - 3), (K, 1))
    y = ttt.ttt_i8_project(o, xs, w[:, 1:K - 2], ws)
    assert torch.equal(y[cut:], ttt.ttt_i8_project(o[cut:], xs[cut:], w[:, 1:K - 2], ws))
    del x, o, y
    # outputs
    N, M = 4096, (1 << 19) + (1 << 16)
    a, s = torch.randint(-128, 128, (M, 64), dtype=I8, device="cuda"), torch.rand(M, device="cuda")
    w, ws = torch.randint(-128, 128, (N, 64), dtype=I8, device="cuda"), torch.rand(N, device="cuda")
    y = ttt.ttt_i8_project(a, s, w, ws)
    assert torch.equal(y[M - 200:], ttt.ttt_i8_project(a[M - 200:], s[M - 200:], w, ws))
    # and the quantiser's rows
    f = y[:, :4000]
    q, sc = ttt.ttt_i8_quantize(f)
    q2, sc2 = ttt.ttt_i8_quantize(f[M - 200:])
    assert torch.equal(q[M - 200:], q2) and torch.equal(sc[M - 200:], sc2)


@pytest.mark.parametrize("name", NAMES)
def test_written_tensors_change_their_version(name):
    fn, outs, ins = _ops(BF, L=40)[name]
    before = [t._version for t in outs], [t._version for t in ins]
    fn(None)
    assert all(t._version > v for t, v in zip(outs, before[0]))
    assert [t._version for t in ins] == before[1]
    with torch.inference_mode():
        _ops(BF, L=40)[name][0](None)


def test_nothing_at_all():
    """Sequences, tokens or features of which there are none."""
    e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device="cuda")
    rate = torch.ones(8, device="cuda")
    h = torch.randn(3, 8, device="cuda")
    y, so = ttt.ttt_lru_forward(e(3, 0, 8), e(3, 0, 8), rate, e(3, 0, 8), h)
    assert y.shape == (3, 0, 8) and torch.equal(so, h)
    _, so = ttt.ttt_lru_forward(e(3, 0, 8), e(3, 0, 8))
    assert not bool(so.any())
    y, so = ttt.ttt_lru_forward(e(0, 5, 8), e(0, 5, 8), rate)
    assert y.shape == (0, 5, 8) and so.shape == (0, 8)
    assert ttt.ttt_lru_step(e(0, 8), e(0, 8), torch.empty(0, 8, device="cuda")).shape == (0, 8)
    g = ttt.ttt_lru_backward(e(3, 0, 8), e(3, 0, 8), e(3, 0, 8), rate, e(3, 0, 8), h, 2 * h)
    assert torch.equal(g["dstate"], 2 * h) and not bool(g["drate"].any())
    g = ttt.ttt_lru_backward(e(0, 4, 8), e(0, 4, 8), e(0, 4, 8), rate)
    assert not bool(g["drate"].any())
    # sequences of no tokens beside others
    x, r = torch.randn(2, 70, 8, device="cuda"), torch.randn(2, 70, 8, device="cuda")
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    y, so = ttt.ttt_lru_forward(x, r, rate, state=h[:2], lens=none)
    assert not bool(y.any()) and torch.equal(so, h[:2])
    g = ttt.ttt_lru_backward(x, r, x, rate, state=h[:2], dstate_out=h[:2], lens=none)
    assert not bool(g["dx"].any()) and not bool(g["dr"].any()) and not bool(g["drate"].any()) and torch.equal(g["dstate"], h[:2])
    q, s = ttt.ttt_i8_quantize(e(0, 16))
    assert q.shape == (0, 16) and s.shape == (0,)
    w, ws = torch.zeros(4, 16, dtype=I8, device="cuda"), torch.zeros(4, device="cuda")
    assert ttt.ttt_i8_linear(e(0, 16), w, ws).shape == (0, 4)
    assert ttt.ttt_i8_linear(torch.zeros(5, 16, dtype=BF, device="cuda"), w[:0], ws[:0]).shape == (5, 0)
    assert ttt.ttt_i8_project(q, s, w, ws).shape == (0, 4)
