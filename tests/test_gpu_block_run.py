"""The operators around the layer as a model runs them: one block (norm, input
projection, convolution, scan, output projection, norm) over ragged prompts,
then token by token, and its training step; on side streams, two calls at
once, captured into graphs and replayed; rows past 4 GiB; and what the Python
binding refuses."""
import pytest
import torch

from tests import block_ref as R
from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def _model(dm, H, P, G, N, K, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    C = H * P + 2 * G * N
    return {"dims": (dm, H, P, G, N, K, C), "post": (1 + 0.1 * r(dm)).cuda(), "pre": (1 + 0.1 * r(dm)).cuda(),
            "scale": (1 + 0.1 * r(dm)).cuda(), "w_in": (r(dm, C + H + dm) * dm ** -0.5).to(dt).cuda(),
            "w_out": (r(H * P, dm) * (H * P) ** -0.5).to(dt).cuda(), "conv_w": (r(C, K) * K ** -0.5).cuda(),
            "conv_b": (0.1 * r(C)).cuda(), "A": -torch.exp(2 * torch.rand(H, generator=g)).cuda(),
            "D": (1 + 0.1 * r(H)).cuda(), "dt_bias": (r(H) - 3).cuda()}


def _split(m, xbc):
    dm, H, P, G, N, K, C = m["dims"]
    return (xbc[..., :H * P].unflatten(-1, (H, P)), xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N)),
            xbc[..., H * P + G * N:].unflatten(-1, (G, N)))


def _block(m, resid, y, conv_state, ssm_state, lens=None):
    """One block over a prompt: (resid, next block's y, conv state, scan state)."""
    dm, H, P, G, N, K, C = m["dims"]
    r, x = ttt.ttt_block_norm(resid, y, m["post"], m["pre"], scale=m["scale"], eps=EPS, lens=lens)
    z = x @ m["w_in"]
    xbc, cs = ttt.ttt_conv_forward(z[..., :C], m["conv_w"], m["conv_b"], conv_state, lens=lens)
    xs, Bm, Cm = _split(m, xbc)
    o, ss = ttt.ttt_ssm_forward(xs, z[..., C:C + H], m["A"], Bm, Cm, m["D"], m["dt_bias"], ssm_state, lens)
    out = o.flatten(2) @ m["w_out"]
    r2, x2 = ttt.ttt_block_norm(r, out, m["post"], m["pre"], gate=z[..., C + H:], gate_act="sigmoid", eps=EPS, lens=lens)
    return r2, x2, cs, ss


def _block_step(m, resid, y, cs, ss):
    dm, H, P, G, N, K, C = m["dims"]
    r, x = ttt.ttt_block_norm(resid[:, None], y[:, None], m["post"], m["pre"], scale=m["scale"], eps=EPS)
    z = x[:, 0] @ m["w_in"]
    xbc = ttt.ttt_conv_step(z[:, :C], m["conv_w"], cs, m["conv_b"])
    xs, Bm, Cm = _split(m, xbc)
    o = ttt.ttt_ssm_step(xs, z[:, C:C + H], m["A"], Bm, Cm, ss, m["D"], m["dt_bias"])
    out = o.flatten(1) @ m["w_out"]
    r2, x2 = ttt.ttt_block_norm(r, out[:, None], m["post"], m["pre"], gate=z[:, None, C + H:], gate_act="sigmoid", eps=EPS)
    return r2[:, 0], x2[:, 0]


def _ref_block(m, resid, y, conv_state, ssm_state, lens):
    dm, H, P, G, N, K, C = m["dims"]
    w = {k: R.t64(v) for k, v in m.items() if k != "dims"}
    r, x = R.block_norm(resid, y, w["post"], w["pre"], None, w["scale"], None, None, "rms", "none", EPS, lens)
    z = x @ w["w_in"]
    xbc, cs = R.conv(z[..., :C], w["conv_w"], w["conv_b"], conv_state, "silu", lens)
    xs, Bm, Cm = _split(m, xbc)
    o, ss = R.scan(xs, z[..., C:C + H], w["A"], Bm, Cm, w["D"], w["dt_bias"], ssm_state, lens)
    r2, x2 = R.block_norm(r, o.flatten(2) @ w["w_out"], w["post"], w["pre"], z[..., C + H:], None, None, None, "rms",
                          "sigmoid", EPS, lens)
    return r2, x2, cs, ss


@pytest.mark.parametrize("dt,rel", [(F32, 2e-5), (BF, 6e-2)])
def test_a_block_over_ragged_prompts_and_then_token_by_token(dt, rel):
    """Against the same chain in 64 bits, relative to each output's largest
    value. fp32: five operators of at most some 100 half steps (6e-8) each and
    two products over 64 and 128 terms. bf16: six roundings to bf16 (2^-8
    each) on the way, the norms' and the gate's factors up to about 2."""
    m = _model(64, 2, 64, 1, 64, 4, dt)
    B, L, T = 3, 90, 4
    lens = torch.tensor([90, 1, 57], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(9)
    resid = torch.randn(B, L + T, 64, generator=g).to(dt).cuda()
    y = torch.randn(B, L + T, 64, generator=g).to(dt).cuda()
    r, x, cs, ss = _block(m, resid[:, :L], y[:, :L], None, None, lens)
    want = _ref_block(m, R.t64(resid[:, :L]), R.t64(y[:, :L]), None, None, lens)
    for got, ref, name in zip((r, x, cs, ss), want, ("resid", "x", "conv state", "state")):
        err = float((R.t64(got) - ref).abs().max() / ref.abs().max())
        print(f"[block] {name}: {err:.1e}", flush=True)
        assert err <= rel, name
    # each sequence goes on from its own length
    rows = torch.cat([torch.cat([resid[b:b + 1, :n], resid[b:b + 1, L:]], 1) if n == L else
                      torch.cat([resid[b:b + 1, :n], resid[b:b + 1, L:], resid[b:b + 1, n:L]], 1)
                      for b, n in enumerate(lens.tolist())])
    ys = torch.cat([torch.cat([y[b:b + 1, :n], y[b:b + 1, L:], y[b:b + 1, n:L]], 1) for b, n in enumerate(lens.tolist())])
    whole = _ref_block(m, R.t64(rows), R.t64(ys), None, None, (lens.cpu() + T))
    for t in range(T):
        r1, x1 = _block_step(m, resid[:, L + t], y[:, L + t], cs, ss)
        for got, ref, name in ((r1, whole[0], "resid"), (x1, whole[1], "x")):
            ref = torch.stack([ref[b, n + t] for b, n in enumerate(lens.tolist())])
            err = float((R.t64(got) - ref).abs().max() / ref.abs().max())
            assert err <= rel, (name, t, err)


def test_a_training_step_of_a_block():
    """The block's gradients by its operators' backwards, in fp32, against
    torch's differentiation of the chain in 64 bits and, along a random
    direction, against central differences of that chain."""
    m = _model(32, 2, 16, 1, 16, 3, F32, 3)
    dm, H, P, G, N, K, C = m["dims"]
    B, L = 2, 40
    g = torch.Generator().manual_seed(4)
    resid, y, dr, dx = (torch.randn(B, L, dm, generator=g).cuda() for _ in range(4))
    # forwards, keeping what the backward passes read
    r, x = ttt.ttt_block_norm(resid, y, m["post"], m["pre"], scale=m["scale"], eps=EPS)
    z = x @ m["w_in"]
    xbc, _ = ttt.ttt_conv_forward(z[..., :C], m["conv_w"], m["conv_b"])
    xs, Bm, Cm = _split(m, xbc)
    scan = (xs, z[..., C:C + H], m["A"], Bm, Cm)
    o, _ = ttt.ttt_ssm_forward(*scan, m["D"], m["dt_bias"])
    out = o.flatten(2) @ m["w_out"]
    gate = z[..., C + H:]
    # backwards
    b2 = ttt.ttt_block_norm_backward(r, out, m["post"], m["pre"], dr, dx, gate=gate, gate_act="sigmoid", eps=EPS)
    do = (b2["dy"] @ m["w_out"].t()).unflatten(-1, (H, P))
    dxbc = torch.empty_like(xbc)
    gx, gB, gC = _split(m, dxbc)
    dz = torch.empty_like(z)
    bs = ttt.ttt_ssm_backward(*scan, do, m["D"], m["dt_bias"], grads={
        "dx": gx, "dB": gB, "dC": gC, "ddt": dz[..., C:C + H], "dA": torch.empty_like(m["A"]),
        "dD": torch.empty_like(m["D"]), "ddt_bias": torch.empty_like(m["A"])})
    bc = ttt.ttt_conv_backward(z[..., :C], m["conv_w"], dxbc, m["conv_b"], grads={
        "dx": dz[..., :C], "dweight": torch.empty_like(m["conv_w"]), "dbias": torch.empty_like(m["conv_b"])})
    dz[..., C + H:] = b2["dgate"]
    b1 = ttt.ttt_block_norm_backward(resid, y, m["post"], m["pre"], b2["dresid"], dz @ m["w_in"].t(), scale=m["scale"],
                                     eps=EPS)
    got = {"resid": b1["dresid"], "y": b1["dy"], "scale": b1["dscale"], "post": b1["dpost_gamma"] + b2["dpost_gamma"],
           "pre": b1["dpre_gamma"] + b2["dpre_gamma"], "w_in": x.flatten(0, 1).t() @ dz.flatten(0, 1),
           "w_out": o.flatten(0, 1).flatten(1).t() @ b2["dy"].flatten(0, 1), "conv_w": bc["dweight"],
           "conv_b": bc["dbias"], "A": bs["dA"], "D": bs["dD"], "dt_bias": bs["ddt_bias"]}
    leaves = {"resid": R.t64(resid), "y": R.t64(y), **{k: R.t64(v) for k, v in m.items() if k != "dims"}}

    def chain(**v):
        mm = dict(v, dims=m["dims"])
        return _ref_block(mm, v["resid"], v["y"], None, None, None)[:2]

    # leaves of the chain: the reference's own copies must not cut the graph
    keep = R.t64
    try:
        R.t64 = lambda t: t
        go = (keep(dr), keep(dx))
        want = R.gradients(chain, leaves, go)
        d = {k: torch.randn(v.shape, generator=g, dtype=R.F64) for k, v in leaves.items()}
        h = 1e-5
        loss = lambda s: sum(float((o * q).sum()) for o, q in zip(chain(**{k: v + s * d[k] for k, v in leaves.items()}), go))
        along = (loss(h) - loss(-h)) / (2 * h)
    finally:
        R.t64 = keep
    for k, w in want.items():
        err = float((R.t64(got[k]) - w).abs().max() / w.abs().max())
        print(f"[block] d{k}: {err:.1e}", flush=True)
        assert err <= 1e-4, k  # some 1000 half steps of fp32 over the chain and its sums of 80 rows
    have = sum(float((R.t64(got[k]) * d[k]).sum()) for k in want)
    assert abs(have - along) <= 1e-4 * sum(float((want[k] * d[k]).abs().sum()) for k in want)


def _ops(dt=BF, B=2, L=200, H=4, N=64, seed=0):
    """Each entry point with its operands and outputs made beforehand:
    name -> (fn(stream), outputs, operands that may change)."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).cuda()
    C, K, D, P = 136, 4, 768, 64
    ops = {}
    x, w, bias, cs = r(B, L, C).to(dt), r(C, K), r(C), r(B, K - 1, C).to(dt)
    y, cso = torch.empty_like(x), torch.empty_like(cs)
    ops["conv_forward"] = (lambda s: ttt.ttt_conv_forward(x, w, bias, cs, y=y, state_out=cso, stream=s), [y, cso], [x])
    gr = {"dx": torch.empty_like(x), "dweight": torch.empty_like(w), "dbias": torch.empty_like(bias),
          "dstate": torch.empty_like(cs)}
    ws = torch.empty(ttt.ttt_conv_backward_workspace(B, L, C, K), dtype=torch.uint8, device="cuda")
    ops["conv_backward"] = (lambda s: ttt.ttt_conv_backward(x, w, x, bias, cs, cs, workspace=ws, grads=gr, stream=s),
                            list(gr.values()), [x])
    xt, yt, st = r(B, C).to(dt), torch.empty(B, C, dtype=dt, device="cuda"), torch.zeros_like(cs)
    ops["conv_step"] = (lambda s: ttt.ttt_conv_step(xt, w, st, bias, y=yt, stream=s), [yt, st], [xt])
    sx, sdt, A = r(B, L, H, P).to(dt), r(B, L, H).to(dt), -torch.rand(H, device="cuda") - 0.1
    Bm, Cm, Dh, s0 = r(B, L, 1, N).to(dt), r(B, L, 1, N).to(dt), r(H), r(B, H, N, P)
    sy, so = torch.empty_like(sx), torch.empty_like(s0)
    ws2 = torch.empty(ttt.ttt_ssm_forward_workspace(B, L, H, P, 1, N), dtype=torch.uint8, device="cuda")
    ops["ssm_forward"] = (lambda s: ttt.ttt_ssm_forward(sx, sdt, A, Bm, Cm, Dh, Dh, s0, y=sy, state_out=so, workspace=ws2,
                                                        stream=s), [sy, so], [sx, sdt])
    sg = {"dx": torch.empty_like(sx), "ddt": torch.empty_like(sdt), "dA": torch.empty_like(A), "dB": torch.empty_like(Bm),
          "dC": torch.empty_like(Cm), "dD": torch.empty_like(A), "ddt_bias": torch.empty_like(A),
          "dstate": torch.empty_like(s0)}
    ws3 = torch.empty(ttt.ttt_ssm_backward_workspace(B, L, H, P, 1, N), dtype=torch.uint8, device="cuda")
    ops["ssm_backward"] = (lambda s: ttt.ttt_ssm_backward(sx, sdt, A, Bm, Cm, sx, Dh, Dh, s0, s0, workspace=ws3, grads=sg,
                                                          stream=s), list(sg.values()), [sx, sdt])
    ty, ts = torch.empty(B, H, P, dtype=dt, device="cuda"), torch.zeros_like(s0)
    ops["ssm_step"] = (lambda s: ttt.ttt_ssm_step(sx[:, 0], sdt[:, 0], A, Bm[:, 0], Cm[:, 0], ts, Dh, Dh, y=ty, stream=s),
                       [ty, ts], [sx])
    n, res, gam, gate = r(B, L, D).to(dt), r(B, L, D), r(D), r(B, L, D).to(dt)
    ro, xo = torch.empty_like(res), torch.empty_like(n)
    ops["block_norm"] = (lambda s: ttt.ttt_block_norm(res, n, gam, gam, gate=gate, scale=gam, gate_act="silu", resid_out=ro,
                                                      x=xo, stream=s), [ro, xo], [n])
    ng = {"dresid": torch.empty_like(res), "dy": torch.empty_like(n), "dgate": torch.empty_like(n), "dscale": torch.empty_like(gam),
          "dpost_gamma": torch.empty_like(gam), "dpre_gamma": torch.empty_like(gam)}
    ws4 = torch.empty(ttt.ttt_block_norm_backward_workspace(B, L, D, 3), dtype=torch.uint8, device="cuda")
    ops["block_norm_backward"] = (lambda s: ttt.ttt_block_norm_backward(res, n, gam, gam, res, n, gate=gate, scale=gam,
                                                                        gate_act="silu", workspace=ws4, grads=ng, stream=s),
                                  list(ng.values()), [n])
    return ops


NAMES = ["conv_forward", "conv_backward", "conv_step", "ssm_forward", "ssm_backward", "ssm_step", "block_norm",
         "block_norm_backward"]
IN_PLACE = ("conv_step", "ssm_step")


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", NAMES)
def test_repeats_bit_for_bit_and_on_a_side_stream(name, dt):
    fn, outs, _ = _ops(dt)[name]

    def run(stream):
        for o in outs:
            o.zero_() if name in IN_PLACE else o.fill_(3)
        torch.cuda.synchronize()
        fn(stream)
        torch.cuda.synchronize()
        return [o.clone() for o in outs]

    a, b, c = run(None), run(None), run(torch.cuda.Stream())
    for u, v, w in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, w)


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name):
    """A graph's replays, with new operands and eager work between them, give
    the eager call's bits each time."""
    fn, outs, ins = _ops(BF)[name]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fn(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn(None)
    for rep in range(3):
        for t in ins:
            t.copy_(torch.roll(t, 1, 0) * 0.75 + 0.25)
        for o in outs:
            o.zero_()
        fn(None)
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_() if name in IN_PLACE else o.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), rep
        torch.randn(1 << 16, device="cuda").sum().item()  # eager work of the program's own


@pytest.mark.parametrize("name", ["ssm_forward", "ssm_backward", "conv_backward", "block_norm_backward"])
def test_two_calls_at_once(name):
    """Two streams, each with its own workspace and outputs."""
    a, b = _ops(BF, L=1500, seed=1)[name], _ops(BF, L=1500, seed=2)[name]
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


def test_rows_past_4_gib_convolution_and_norm():
    """Tokens whose offsets pass 2^31 elements: the tail equals that of a short
    call over the same rows."""
    B, C, K = 1, 2176, 4
    L = (1 << 20) + 37  # 2.3e9 elements
    x = torch.empty(B, L, C, device="cuda", dtype=BF)
    for i in range(0, L, 1 << 17):
        x[:, i:i + (1 << 17)].normal_()
    w, b = torch.randn(C, K, device="cuda"), torch.randn(C, device="cuda")
    y, so = ttt.ttt_conv_forward(x, w, b)
    cut = L - 100
    y2, so2 = ttt.ttt_conv_forward(x[:, cut:], w, b, x[:, cut - K + 1:cut].contiguous())
    assert torch.equal(y[:, cut:], y2) and torch.equal(so, so2)
    g = torch.randn(C, device="cuda")
    r, n = ttt.ttt_block_norm(x, y, g, g)
    r2, n2 = ttt.ttt_block_norm(x[:, cut:], y[:, cut:], g, g)
    assert torch.equal(r[:, cut:], r2) and torch.equal(n[:, cut:], n2)
    del r, n
    d = ttt.ttt_conv_backward(x, w, y, b)["dx"]
    d2 = ttt.ttt_conv_backward(x[:, cut:], w, y[:, cut:], b, x[:, cut - K + 1:cut].contiguous())["dx"]
    assert torch.equal(d[:, cut:], d2)


def test_rows_past_4_gib_scan():
    """The same of the scan, whose state before the tail comes from a call over
    the rows before it; the tail's first and last rows and the state."""
    B, H, P, N = 1, 32, 64, 64
    L = (1 << 20) + 70
    x = torch.empty(B, L, H, P, device="cuda", dtype=BF)
    for i in range(0, L, 1 << 17):
        x[:, i:i + (1 << 17)].normal_()
    Bm, Cm = (torch.randn(B, L, 1, N, device="cuda").mul_(0.1).to(BF) for _ in range(2))
    dt = torch.randn(B, L, H, device="cuda").sub_(3).to(BF)
    A = -torch.rand(H, device="cuda") - 0.5
    y, so = ttt.ttt_ssm_forward(x, dt, A, Bm, Cm)
    cut = (1 << 20) - 64 * 5
    _, st = ttt.ttt_ssm_forward(x[:, :cut], dt[:, :cut], A, Bm[:, :cut], Cm[:, :cut])
    y2, so2 = ttt.ttt_ssm_forward(x[:, cut:], dt[:, cut:], A, Bm[:, cut:], Cm[:, cut:], state=st)
    scale = float(y2.float().abs().max())
    # two bf16 operand roundings of the same terms, cut into other segments
    assert float((y[:, cut:].float() - y2.float()).abs().max()) <= 4 * 2.0 ** -8 * scale
    assert float((so - so2).abs().max()) <= 1e-4 * float(so2.abs().max())


def test_python_refusals():
    x = torch.zeros(2, 5, 8, device="cuda", dtype=BF)
    w = torch.zeros(8, 4, device="cuda")
    st = torch.zeros(2, 3, 8, device="cuda", dtype=BF)
    ok = lambda **k: ttt.ttt_conv_forward(**{"x": x, "weight": w, "state": st, **k})
    ok()
    with pytest.raises(ValueError, match="device tensor"):
        ok(x=x.cpu())
    with pytest.raises(TypeError, match="not supported"):
        ok(x=x.half())
    with pytest.raises(TypeError, match="dtype"):
        ok(weight=w.to(BF))
    with pytest.raises(ValueError, match="shape"):
        ok(weight=w[:4])
    with pytest.raises(ValueError, match="is on cpu"):
        ok(weight=w.cpu())
    with pytest.raises(ValueError, match="innermost"):
        ok(x=torch.zeros(2, 8, 5, device="cuda", dtype=BF).transpose(1, 2))
    with pytest.raises(ValueError, match="activation"):
        ok(activation="tanh")
    with pytest.raises(TypeError, match="lens"):
        ok(lens=torch.tensor([1, 2], device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        ok(state=torch.zeros(2, 3, 16, device="cuda", dtype=BF)[..., ::2])
    with pytest.raises(ttt.TTTError, match="overlaps"):
        ok(y=x)
    with pytest.raises(ttt.TTTError, match="K = 5"):
        ttt.ttt_conv_forward(x, torch.zeros(8, 5, device="cuda"))
    with pytest.raises(ValueError, match="grads"):
        ttt.ttt_conv_backward(x, w, x, grads={"dx": x})
    sx, dt = torch.zeros(1, 4, 2, 8, device="cuda"), torch.zeros(1, 4, 2, device="cuda")
    A, Bm = torch.zeros(2, device="cuda"), torch.zeros(1, 4, 1, 8, device="cuda")
    ttt.ttt_ssm_forward(sx, dt, A, Bm, Bm)
    with pytest.raises(TypeError, match="dt"):
        ttt.ttt_ssm_forward(sx, dt.to(BF), A, Bm, Bm)
    with pytest.raises(ValueError, match="state"):
        ttt.ttt_ssm_step(sx[:, 0], dt[:, 0], A, Bm[:, 0], Bm[:, 0], torch.zeros(1, 2, 8, 9, device="cuda"))
    with pytest.raises(ValueError, match="gate has"):
        ttt.ttt_block_norm(x, x, gate=torch.zeros(1, device="cuda")[0])
    with pytest.raises(ValueError, match="norm"):
        ttt.ttt_block_norm(x, x, norm="batch")
    with pytest.raises(ttt.TTTError, match="workspace"):
        ttt.ttt_conv_backward(x, w, torch.zeros_like(x), workspace=torch.empty(16, device="cuda", dtype=torch.uint8))


def test_lengths_are_clamped():
    """Lengths below 0 and past L act as 0 and L."""
    d = torch.randn(3, 70, 2, 64, device="cuda").to(BF)
    dt = torch.randn(3, 70, 2, device="cuda").to(BF)
    A, Bm = -torch.rand(2, device="cuda"), torch.randn(3, 70, 1, 64, device="cuda").to(BF)
    wild = torch.tensor([-5, 1 << 30, 33], dtype=torch.int32, device="cuda")
    tame = torch.tensor([0, 70, 33], dtype=torch.int32, device="cuda")
    for f in (lambda n: ttt.ttt_ssm_forward(d, dt, A, Bm, Bm, lens=n),
              lambda n: tuple(ttt.ttt_ssm_backward(d, dt, A, Bm, Bm, d, lens=n).values()),
              lambda n: ttt.ttt_conv_forward(d.flatten(2), torch.ones(128, 3, device="cuda"), lens=n),
              lambda n: tuple(ttt.ttt_conv_backward(d.flatten(2), torch.ones(128, 3, device="cuda"), d.flatten(2), lens=n).values()),
              lambda n: ttt.ttt_block_norm(d.flatten(2), d.flatten(2), lens=n)):
        for a, b in zip(f(wild), f(tame)):
            assert torch.equal(a, b)
