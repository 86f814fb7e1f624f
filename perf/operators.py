"""What is measured of the operators around a recurrent layer block: the short
causal convolution, the selective state space scan and the block norm, each in
the directions that a prompt, a single token and a training step take.

Shapes follow bench.py: d_model 768 (12 heads of 64) and 2048 (32 heads of
64), contexts of 2048, 8192 and 32768 tokens, 64 sequences in decode. The
convolution runs over the heads' features and the scan's B and C together, as
one slice of an input projection's output.
"""
import torch

own = False

# cases -----------------------------------------------------------------------


def _conv(name, direction, B, L, C, K, dtype, ragged=False, state=False, act="silu", bias=True):
    c = {"op": "conv", "dir": direction, "B": B, "L": L, "C": C, "K": K, "dtype": dtype,
         "ragged": ragged, "state": state, "act": act, "bias": bias}
    return {"name": name, **c} if name else c


def _scan(name, direction, B, L, H, P, G, N, dtype, ragged=False, state=False):
    c = {"op": "scan", "dir": direction, "B": B, "L": L, "H": H, "P": P, "G": G, "N": N,
         "dtype": dtype, "ragged": ragged, "state": state}
    return {"name": name, **c} if name else c


def _norm(name, direction, B, L, D, dtype, resid, kind="rms", gate="token", act="sigmoid",
          scale=True, ragged=False):
    c = {"op": "norm", "dir": direction, "B": B, "L": L, "D": D, "dtype": dtype, "resid": resid,
         "kind": kind, "gate": gate, "act": act, "scale": scale, "ragged": ragged}
    return {"name": name, **c} if name else c


def listed():
    return [
        # prefill of two 8k prompts at width 2048, one group of B and C of 64 each
        _conv("conv_prompt_8k", "prompt", 2, 8192, 2176, 4, "bf16"),
        # continued prompts of unequal length, a channel count that no vector divides
        _conv("conv_prompt_ragged", "prompt", 3, 1037, 771, 3, "f32", ragged=True, state=True),
        # one token for each of 64 sequences
        _conv("conv_step_64", "step", 64, 1, 2176, 4, "bf16", state=True),
        # a training step at width 768
        _conv("conv_backward_2k", "backward", 4, 2048, 896, 4, "bf16"),
        # the same prefill's scan
        _scan("scan_prompt_8k", "prompt", 2, 8192, 32, 64, 1, 64, "bf16"),
        # one long prompt with a wide state
        _scan("scan_prompt_32k", "prompt", 1, 32768, 32, 64, 1, 128, "bf16"),
        # continued prompts of unequal length in fp32, odd sizes, two groups
        _scan("scan_prompt_ragged", "prompt", 3, 517, 6, 48, 2, 24, "f32", ragged=True, state=True),
        # one token for each of 64 sequences
        _scan("scan_step_64", "step", 64, 1, 32, 64, 1, 64, "bf16", state=True),
        # a training step at width 768
        _scan("scan_backward_2k", "backward", 4, 2048, 12, 64, 1, 64, "bf16"),
        # between two blocks of the 8k prefill, residual stream in fp32
        _norm("norm_prompt_8k", "prompt", 2, 8192, 2048, "bf16", "f32"),
        # between two blocks for a single token: latency
        _norm("norm_step_1", "prompt", 1, 1, 768, "bf16", "bf16", gate="channel", act="tanh"),
        # a training step at width 768
        _norm("norm_backward_2k", "backward", 4, 2048, 768, "bf16", "bf16", kind="layer"),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    import math
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv", "scan", "scan", "scan", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "conv":
        d = rng.choice(["prompt", "step", "backward"])
        C = rng.choice([896, 2176, _log(rng, 16, 4352), _log(rng, 2, 544) * 8])
        B = _log(rng, 1, 512) if d == "step" else _log(rng, 1, 16)
        L = 1 if d == "step" else _log(rng, 2, max(2, min(32768, 35_000_000 // (B * C))))
        return _conv("", d, B, L, C, rng.choice([2, 3, 4, 4]), dtype,
                     d != "step" and rng.random() < 0.4, d == "step" or rng.random() < 0.4,
                     rng.choice(["silu", "silu", "none"]), rng.random() < 0.7)
    if op == "scan":
        d = rng.choice(["prompt", "prompt", "step", "backward"])
        P = rng.choice([64, 64, 64, 16, rng.randint(1, 64)])
        N = rng.choice([64, 128, 16, 32, rng.randint(1, 128)])
        G = rng.choice([1, 1, 2, 4])
        H = G * _log(rng, 1, 32 // G)
        B = _log(rng, 1, 256) if d == "step" else _log(rng, 1, 16)
        most = 8_000_000_000 if d == "prompt" else 1_600_000_000
        L = 1 if d == "step" else _log(rng, 2, max(2, min(32768, most // (B * H * P * max(N, 32)))))
        return _scan("", d, B, L, H, P, G, N, dtype, d != "step" and rng.random() < 0.4,
                     d == "step" or rng.random() < 0.4)
    d = rng.choice(["prompt", "backward"])
    D = rng.choice([768, 2048, _log(rng, 16, 8192), _log(rng, 2, 1024) * 8])
    B = _log(rng, 1, 64)
    L = _log(rng, 1, max(1, min(32768, 33_000_000 // (B * D))))
    return _norm("", d, B, L, D, dtype, rng.choice([dtype, "f32"]), rng.choice(["rms", "layer"]),
                 rng.choice(["token", "sequence", "channel", "no"]),
                 rng.choice(["none", "sigmoid", "silu", "tanh"]), rng.random() < 0.6,
                 L > 1 and rng.random() < 0.4)


# inputs ----------------------------------------------------------------------

_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lens(case, r):
    """Lengths from none at all to the whole of L, the longest always whole."""
    if not case["ragged"]:
        return None
    n = torch.randint(0, case["L"] + 1, (case["B"],), generator=r, device="cuda", dtype=torch.int32)
    n[0] = case["L"]
    return n


def prepare(case, seed):
    r = torch.Generator(device="cuda")
    r.manual_seed(seed)
    io = _TYPE[case["dtype"]]

    def normal(*shape, dtype=io, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=r, device="cuda") * std + mean).to(dtype)

    f32 = torch.float32
    B, L = case["B"], case["L"]
    s = {"case": dict(case), "lens": _lens(case, r)}
    if case["op"] == "conv":
        C, K = case["C"], case["K"]
        # a slice of the input projection's output: the gate's features lie beside it
        row = C + 8 * (C // 16)
        s["x"] = normal(B, row)[:, row - C:] if case["dir"] == "step" else normal(B, L, row)[..., row - C:]
        s["weight"] = normal(C, K, dtype=f32, std=K ** -0.5)
        s["bias"] = normal(C, dtype=f32, std=0.1) if case["bias"] else None
        s["state"] = normal(B, K - 1, C) if case["state"] else None
        if case["dir"] == "backward":
            s["dy"] = normal(B, L, C)
            s["dstate_out"] = normal(B, K - 1, C) if case["state"] else None
    elif case["op"] == "scan":
        H, P, G, N = case["H"], case["P"], case["G"], case["N"]
        one = case["dir"] == "step"
        lead = (B,) if one else (B, L)
        # x, B and C: three slices of the convolution's output
        xbc = torch.nn.functional.silu(normal(*lead, H * P + 2 * G * N, dtype=f32, std=1.5)).to(io)
        s["x"] = xbc[..., :H * P].unflatten(-1, (H, P))
        s["B"] = xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N))
        s["C"] = xbc[..., H * P + G * N:].unflatten(-1, (G, N))
        s["dt"] = normal(*lead, H)
        s["A"] = -torch.exp(torch.rand(H, generator=r, device="cuda") * 2.77)  # -1 .. -16
        s["D"] = normal(H, dtype=f32, std=0.3, mean=1.0)
        # softplus(dt + dt_bias) around 0.001 .. 0.1, as such layers are initialised
        s["dt_bias"] = torch.log(torch.expm1(torch.exp(
            torch.rand(H, generator=r, device="cuda") * 4.6 - 6.9)))
        s["state"] = normal(B, H, N, P, dtype=f32) if case["state"] else None
        if case["dir"] == "backward":
            s["dy"] = normal(B, L, H, P)
            s["dstate_out"] = normal(B, H, N, P, dtype=f32) if case["state"] else None
    else:
        D, rt = case["D"], _TYPE[case["resid"]]
        s["resid"] = normal(B, L, D, dtype=rt, std=2.0)
        s["y"] = normal(B, L, D, std=0.5)
        shape = {"token": (B, L, D), "sequence": (B, D), "channel": (D,)}.get(case["gate"])
        s["gate"] = None if shape is None else normal(*shape, dtype=io if case["gate"] == "token" else f32)
        s["scale"] = normal(D, dtype=f32, std=0.1, mean=1.0) if case["scale"] else None
        for k in ("post", "pre"):
            s[k + "_gamma"] = normal(D, dtype=f32, std=0.1, mean=1.0)
            s[k + "_beta"] = normal(D, dtype=f32, std=0.1) if case["kind"] == "layer" else None
        if case["dir"] == "backward":
            s["dresid_out"] = normal(B, L, D, dtype=rt)
            s["dx"] = normal(B, L, D)
    return s


def run(s):
    c = s["case"]
    if own:
        return _own(s)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[c["op"]](s, c)


def _own(s):
    from test_sequence_layer_ttt_amd import ttt
    c = s["case"]
    if c["op"] == "conv":
        kw = {"bias": s["bias"], "activation": c["act"]}
        if c["dir"] == "prompt":
            return ttt.ttt_conv_forward(s["x"], s["weight"], state=s["state"], lens=s["lens"], **kw)
        if c["dir"] == "step":
            return ttt.ttt_conv_step(s["x"], s["weight"], s["state"], **kw), s["state"]
        return ttt.ttt_conv_backward(s["x"], s["weight"], s["dy"], state=s["state"],
                                     dstate_out=s["dstate_out"], lens=s["lens"], **kw)
    if c["op"] == "scan":
        args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
        kw = {"D": s["D"], "dt_bias": s["dt_bias"]}
        if c["dir"] == "prompt":
            return ttt.ttt_ssm_forward(*args, state=s["state"], lens=s["lens"], **kw)
        if c["dir"] == "step":
            return ttt.ttt_ssm_step(*args, s["state"], **kw), s["state"]
        return ttt.ttt_ssm_backward(*args, s["dy"], state=s["state"], dstate_out=s["dstate_out"],
                                    lens=s["lens"], **kw)
    kw = {"gate": s["gate"], "scale": s["scale"], "post_beta": s["post_beta"],
          "pre_beta": s["pre_beta"], "norm": c["kind"], "gate_act": c["act"], "lens": s["lens"]}
    if c["dir"] == "prompt":
        return ttt.ttt_block_norm(s["resid"], s["y"], s["post_gamma"], s["pre_gamma"], **kw)
    return ttt.ttt_block_norm_backward(s["resid"], s["y"], s["post_gamma"], s["pre_gamma"],
                                       s["dresid_out"], s["dx"], **kw)


# plain forms -----------------------------------------------------------------


def _rows(s, L):
    """[B,L,1] truth values: the rows within each sequence's length; None if all are."""
    if s["lens"] is None:
        return None
    return (torch.arange(L, device="cuda")[None] < s["lens"][:, None])[..., None]


def _keep(v, rows):
    if rows is None or v is None:
        return v
    return torch.where(rows.reshape(rows.shape[:2] + (1,) * (v.dim() - 2)), v, torch.zeros((), device=v.device, dtype=v.dtype))


def _drop_none(d):
    return {k: v for k, v in d.items() if v is not None}


def _plain_conv(s, c):
    x, w, K, io = s["x"], s["weight"], c["K"], s["x"].dtype
    B, C = x.shape[0], x.shape[-1]
    if c["dir"] == "step":
        taps = torch.cat([s["state"].float(), x.float()[:, None]], 1)  # [B,K,C]
        z = (taps * w.t()).sum(1)
        z = z if s["bias"] is None else z + s["bias"]
        s["state"].copy_(taps[:, 1:])
        return (z * torch.sigmoid(z) if c["act"] == "silu" else z).to(io), s["state"]
    L, rows = x.shape[1], _rows(s, x.shape[1])
    head = torch.zeros(B, K - 1, C, device="cuda") if s["state"] is None else s["state"].float()
    full = torch.cat([head, _keep(x.float(), rows)], 1)  # [B,K-1+L,C]
    taps = full.unfold(1, K, 1)  # [B,L,C,K]
    z = (taps * w).sum(-1)
    z = z if s["bias"] is None else z + s["bias"]
    n = torch.full((B,), L, device="cuda") if s["lens"] is None else s["lens"].long()
    last = n[:, None] + torch.arange(K - 1, device="cuda")  # rows of `full` that the state holds
    at = last[..., None].expand(-1, -1, C)
    sig = torch.sigmoid(z)
    if c["dir"] == "prompt":
        y = _keep(z * sig if c["act"] == "silu" else z, rows)
        return y.to(io), torch.gather(full, 1, at).to(io)
    dz = s["dy"].float()
    dz = _keep(dz * sig * (1 + z * (1 - sig)) if c["act"] == "silu" else dz, rows)
    behind = torch.cat([dz.new_zeros(B, K - 1, C), dz, dz.new_zeros(B, K - 1, C)], 1)
    dfull = (behind.unfold(1, K, 1) * w.flip(1)).sum(-1)  # [B,K-1+L,C]
    if s["dstate_out"] is not None:
        dfull = dfull.scatter_add(1, at, s["dstate_out"].float())
    return _drop_none({
        "dx": _keep(dfull[:, K - 1:], rows).to(io),
        "dweight": (dz[..., None] * taps).sum((0, 1)),
        "dbias": None if s["bias"] is None else dz.sum((0, 1)),
        "dstate": None if s["state"] is None else dfull[:, :K - 1].to(io)})


def _softplus(z):
    return torch.clamp(z, min=0) + torch.log1p(torch.exp(-z.abs()))


def _plain_scan(s, c):
    io, H, P, G, N = s["x"].dtype, c["H"], c["P"], c["G"], c["N"]
    z = s["dt"].float() + s["dt_bias"]
    if c["dir"] == "step":
        dt = _softplus(z)
        Bh = s["B"].float().repeat_interleave(H // G, 1)
        Ch = s["C"].float().repeat_interleave(H // G, 1)
        x = s["x"].float()
        s["state"].mul_(torch.exp(dt * s["A"])[..., None, None]).add_(Bh[..., None] * (dt[..., None] * x)[:, :, None])
        y = (Ch[..., None] * s["state"]).sum(2) + s["D"][:, None] * x
        return y.to(io), s["state"]
    Bn, L = s["x"].shape[:2]
    rows = _rows(s, L)
    Q = 64
    nc = -(-L // Q)

    def chunks(v):  # [B,L,...] -> [B,heads,nc,Q,...]
        v = _keep(v.float(), rows)
        v = torch.cat([v, v.new_zeros((Bn, nc * Q - L) + v.shape[2:])], 1)
        return v.unflatten(1, (nc, Q)).movedim(3, 1).contiguous()

    def flat(v):  # the inverse
        return _keep(v.movedim(1, 3).flatten(1, 2)[:, :L], rows)

    x, dt = chunks(s["x"]), chunks(_softplus(z))
    Bg, Cg = chunks(s["B"]), chunks(s["C"])
    Bh, Ch = Bg.repeat_interleave(H // G, 1), Cg.repeat_interleave(H // G, 1)
    A = s["A"][:, None, None]
    la = torch.cumsum((dt * A).double(), -1)  # [B,H,nc,Q]: log of the decay since the chunk's start
    low = torch.ones(Q, Q, device="cuda", dtype=torch.bool).tril()
    decay = torch.exp(torch.where(low, la[..., :, None] - la[..., None, :], -torch.inf)).float()
    into, out = torch.exp(la).float(), torch.exp(la[..., -1:] - la).float()
    xt = x * dt[..., None]
    M = (Cg @ Bg.mT.contiguous()).repeat_interleave(H // G, 1) * decay
    # states at the chunks' borders: every chunk's own share, decayed to each later border
    tot = torch.cat([la.new_zeros(Bn, H, 1), torch.cumsum(la[..., -1], -1)], -1)  # [B,H,nc+1]
    between = tot[..., :, None] - tot[..., None, :]
    border = torch.ones(nc + 1, nc + 1, device="cuda", dtype=torch.bool).tril()
    carry = torch.exp(torch.where(border, between, -torch.inf)).float()
    share = Bh.mT.contiguous() @ (xt * out[..., None])  # [B,H,nc,N,P]
    first = share.new_zeros(Bn, H, 1, N, P) if s["state"] is None else s["state"][:, :, None]
    S = (carry @ torch.cat([first, share], 2).flatten(3)).unflatten(3, (N, P))  # [B,H,nc+1,N,P]
    CS = Ch @ S[:, :, :-1]
    D = s["D"][:, None, None, None]
    if c["dir"] == "prompt":
        y = M @ xt + into[..., None] * CS + D * x
        return flat(y).to(io), S[:, :, -1].contiguous()
    dy = chunks(s["dy"])
    share = Ch.mT.contiguous() @ (dy * into[..., None])
    last = share.new_zeros(Bn, H, 1, N, P) if s["dstate_out"] is None else s["dstate_out"][:, :, None]
    dS = (carry.mT.contiguous() @ torch.cat([share, last], 2).flatten(3)).unflatten(3, (N, P))
    BdS = Bh @ dS[:, :, 1:]
    dxt = M.mT.contiguous() @ dy + out[..., None] * BdS
    dM = (dy @ xt.mT.contiguous()) * decay
    dC = dM @ Bh + into[..., None] * (dy @ S[:, :, :-1].mT.contiguous())
    dB = dM.mT.contiguous() @ Ch + out[..., None] * (xt @ dS[:, :, 1:].mT.contiguous())
    W = dM * (Cg @ Bg.mT.contiguous()).repeat_interleave(H // G, 1)
    ends = out * (BdS * xt).sum(-1)
    dla = W.sum(-1) - W.sum(-2) + into * (dy * CS).sum(-1) - ends
    whole = ends.sum(-1) + into[..., -1] * (S[:, :, :-1] * dS[:, :, 1:]).sum((-1, -2))
    da = torch.flip(torch.cumsum(torch.flip(dla, [-1]), -1), [-1]) + whole[..., None]
    ddt = da * A + (x * dxt).sum(-1)
    dz = _keep(flat(ddt) * torch.sigmoid(z), rows)
    return _drop_none({
        "dx": flat(dxt * dt[..., None] + D * dy).to(io), "ddt": dz.to(io),
        "dA": (da * dt).double().sum((0, 2, 3)).float(),
        "dB": flat(dB.unflatten(1, (G, H // G)).sum(2)).to(io),
        "dC": flat(dC.unflatten(1, (G, H // G)).sum(2)).to(io),
        "dD": (dy * x).sum(-1).double().sum((0, 2, 3)).float(),
        "ddt_bias": dz.double().sum((0, 1)).float(),
        "dstate": None if s["state"] is None else dS[:, :, 0].contiguous()})


_EPS = 1e-6


def _plain_gate(s, c):
    """The gate's value and its derivative, over [B,L,D] or broadcast to it."""
    if s["gate"] is None:
        return None, None
    g = s["gate"].float()
    g = g[:, None] if c["gate"] == "sequence" else g
    sig, th = torch.sigmoid(g), torch.tanh(g)
    return {"none": (g, torch.ones_like(g)), "sigmoid": (sig, sig * (1 - sig)),
            "silu": (g * sig, sig * (1 + g * (1 - sig))), "tanh": (th, 1 - th * th)}[c["act"]]


def _plain_hat(u, kind):
    m = u.mean(-1, keepdim=True) if kind == "layer" else 0.0
    r = torch.rsqrt((u - m).square().mean(-1, keepdim=True) + _EPS)
    return (u - m) * r, r


def _plain_unhat(g, hat, r, kind):
    m = g.mean(-1, keepdim=True) if kind == "layer" else 0.0
    return r * (g - m - hat * (g * hat).mean(-1, keepdim=True))


def _plain_norm(s, c):
    kind, io, rt = c["kind"], s["y"].dtype, s["resid"].dtype
    rows = _rows(s, c["L"])
    a, da = _plain_gate(s, c)
    yh, yr = _plain_hat(_keep(s["y"].float(), rows), kind)
    n = yh * s["post_gamma"] if s["post_beta"] is None else yh * s["post_gamma"] + s["post_beta"]
    resid = _keep(s["resid"].float(), rows)
    r = (resid if s["scale"] is None else s["scale"] * resid) + (n if a is None else a * n)
    rh, rr = _plain_hat(r, kind)
    if c["dir"] == "prompt":
        x = rh * s["pre_gamma"] if s["pre_beta"] is None else rh * s["pre_gamma"] + s["pre_beta"]
        return _keep(r, rows).to(rt), _keep(x, rows).to(io)
    dx = _keep(s["dx"].float(), rows)
    dr = _keep(s["dresid_out"].float(), rows) + _plain_unhat(dx * s["pre_gamma"], rh, rr, kind)
    dn = dr if a is None else dr * a
    dgate = None
    if a is not None:
        dgate = _keep(dr * n * da, rows)
        dgate = {"token": lambda: dgate.to(io), "sequence": lambda: dgate.sum(1),
                 "channel": lambda: dgate.sum((0, 1))}[c["gate"]]()
    return _drop_none({
        "dresid": _keep(dr if s["scale"] is None else dr * s["scale"], rows).to(rt),
        "dy": _keep(_plain_unhat(dn * s["post_gamma"], yh, yr, kind), rows).to(io),
        "dgate": dgate,
        "dscale": None if s["scale"] is None else _keep(dr * resid, rows).sum((0, 1)),
        "dpost_gamma": _keep(dn * yh, rows).sum((0, 1)),
        "dpost_beta": None if s["post_beta"] is None else _keep(dn, rows).sum((0, 1)),
        "dpre_gamma": (dx * rh).sum((0, 1)),
        "dpre_beta": None if s["pre_beta"] is None else dx.sum((0, 1))})


# the definitions, in 64 bits ---------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    c = s["case"]
    steps = c["L"]
    s["n"] = [steps] * c["B"] if s["lens"] is None else s["lens"].tolist()
    if c["op"] == "scan":
        if c["dir"] == "backward" and c["B"] * c["H"] * steps * c["N"] * c["P"] > 4e9:
            return None  # every token's state is held
        return _exact_scan(s, c)
    return _exact_conv(s, c) if c["op"] == "conv" else _exact_norm(s, c)


def _exact_conv(s, c):
    """z_t = bias + sum_k w_k x_{t-K+1+k}, one tap at a time."""
    x, w, K, B, L = s["x"], s["weight"], c["K"], c["B"], c["L"]
    if c["dir"] == "step":
        x = x[:, None]
    C = x.shape[-1]
    state = x.new_zeros(B, K - 1, C) if s["state"] is None else s["state"]
    z = x.new_zeros(B, L, C)
    if s["bias"] is not None:
        z += s["bias"]
    for k in range(K):
        back = K - 1 - k  # this tap reads the token `back` before
        if L > back:
            z[:, back:] += w[:, k] * x[:, :L - back]
        m = min(back, L)
        z[:, :m] += w[:, k] * state[:, K - 1 - back:K - 1 - back + m]
    sig = 1 / (1 + torch.exp(-z))
    silu = c["act"] == "silu"
    if c["dir"] != "backward":
        y = z * sig if silu else z
        new = torch.empty_like(state)
        for b, n in enumerate(s["n"]):
            y[b, n:] = 0
            new[b] = torch.cat([state[b], x[b, :n]])[n:]
        return (y[:, 0], new) if c["dir"] == "step" else (y, new)
    dz = s["dy"] * (sig + z * sig * (1 - sig)) if silu else s["dy"].clone()
    for b, n in enumerate(s["n"]):
        dz[b, n:] = 0
    dx, dstate, dw = torch.zeros_like(x), torch.zeros_like(state), torch.zeros_like(w)
    for k in range(K):
        back = K - 1 - k
        if L > back:
            dx[:, :L - back] += w[:, k] * dz[:, back:]
            dw[:, k] += (dz[:, back:] * x[:, :L - back]).sum((0, 1))
        m = min(back, L)
        dstate[:, k:k + m] += w[:, k] * dz[:, :m]
        dw[:, k] += (dz[:, :m] * state[:, k:k + m]).sum((0, 1))
    if s["dstate_out"] is not None:
        for b, n in enumerate(s["n"]):
            for j in range(K - 1):  # the state's row j is row n + j of (state, x)
                i = n + j
                if i < K - 1:
                    dstate[b, i] += s["dstate_out"][b, j]
                else:
                    dx[b, i - K + 1] += s["dstate_out"][b, j]
    for b, n in enumerate(s["n"]):
        dx[b, n:] = 0
    return _drop_none({"dx": dx, "dweight": dw,
                       "dbias": None if s["bias"] is None else dz.sum((0, 1)),
                       "dstate": None if s["state"] is None else dstate})


def _exact_scan(s, c):
    """h_t = exp(dt_t A) h_{t-1} + dt_t B_t x_t, y_t = C_t h_t + D x_t, token by token."""
    B, L, H, P, G, N = (c[k] for k in ("B", "L", "H", "P", "G", "N"))
    one = c["dir"] == "step"
    x, z, Bv, Cv = (s[k][:, None] if one else s[k] for k in ("x", "dt", "B", "C"))
    z = z + s["dt_bias"]
    live = (torch.arange(L, device="cuda")[None] < torch.tensor(s["n"], device="cuda")[:, None])[..., None]
    dt = torch.where(live, torch.logaddexp(z, torch.zeros_like(z)), 0.0)
    A, D = s["A"], s["D"]
    a = torch.exp(dt * A)
    u = dt[..., None] * x
    head = torch.arange(H, device="cuda") // (H // G)
    h = x.new_zeros(B, H, N, P) if s["state"] is None else s["state"].clone()
    h0, kept, y = h, [], torch.empty_like(x)
    for t in range(L):
        h = a[:, t, :, None, None] * h + Bv[:, t, head, :, None] * u[:, t, :, None, :]
        if c["dir"] == "backward":
            kept.append(h)
        else:
            y[:, t] = (Cv[:, t, head, None, :] @ h)[:, :, 0]
    if c["dir"] != "backward":
        y = torch.where(live[..., None], y + D[:, None] * x, 0.0)
        return (y[:, 0], h) if one else (y, h)
    dy = torch.where(live[..., None], s["dy"], 0.0)
    g = torch.zeros_like(h) if s["dstate_out"] is None else s["dstate_out"].clone()
    du, da = torch.empty_like(x), torch.empty_like(dt)
    dB, dC = torch.zeros_like(Bv), torch.zeros_like(Cv)
    for t in reversed(range(L)):
        g = g + Cv[:, t, head, :, None] * dy[:, t, :, None, :]  # the loss's gradient in h_t
        prev = kept[t - 1] if t else h0
        dC[:, t] = (kept[t] @ dy[:, t, :, :, None])[..., 0].unflatten(1, (G, H // G)).sum(2)
        dB[:, t] = (g @ u[:, t, :, :, None])[..., 0].unflatten(1, (G, H // G)).sum(2)
        du[:, t] = (Bv[:, t, head, None, :] @ g)[:, :, 0]
        da[:, t] = (g * prev).sum((-1, -2)) * a[:, t]  # with respect to dt_t A
        g = a[:, t, :, None, None] * g
    ddt = torch.where(live, (da * A + (x * du).sum(-1)) / (1 + torch.exp(-z)), 0.0)
    mask = live[..., None]
    return _drop_none({
        "dx": torch.where(mask, dt[..., None] * du + D[:, None] * dy, 0.0), "ddt": ddt,
        "dA": (da * dt).sum((0, 1)), "dB": torch.where(mask, dB, 0.0),
        "dC": torch.where(mask, dC, 0.0), "dD": (dy * x).sum((0, 1, 3)), "ddt_bias": ddt.sum((0, 1)),
        "dstate": None if s["state"] is None else g})


def _exact_norm(s, c):
    """By the chain rule of the written formula, through torch's differentiation in 64 bits."""
    leaf = {k: s[k].requires_grad_(c["dir"] == "backward") for k in
            ("resid", "y", "gate", "scale", "post_gamma", "post_beta", "pre_gamma", "pre_beta")
            if s[k] is not None}

    def norm(u, which):
        if c["kind"] == "layer":
            u = u - u.mean(-1, keepdim=True)
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + _EPS) * leaf[which + "_gamma"]
        return u + leaf[which + "_beta"] if which + "_beta" in leaf else u

    n = norm(leaf["y"], "post")
    if "gate" in leaf:
        g = leaf["gate"][:, None] if c["gate"] == "sequence" else leaf["gate"]
        n = n * {"none": lambda: g, "sigmoid": lambda: 1 / (1 + torch.exp(-g)),
                 "silu": lambda: g / (1 + torch.exp(-g)), "tanh": lambda: torch.tanh(g)}[c["act"]]()
    r = (leaf["scale"] * leaf["resid"] if "scale" in leaf else leaf["resid"]) + n
    x = norm(r, "pre")
    live = torch.arange(c["L"], device="cuda")[None] < torch.tensor(s["n"], device="cuda")[:, None]
    live = live[..., None].double()
    if c["dir"] == "prompt":
        return r * live, x * live
    loss = (r * live * s["dresid_out"]).sum() + (x * live * s["dx"]).sum()
    return {"d" + k: g for k, g in zip(leaf, torch.autograd.grad(loss, list(leaf.values())))}


# what a pass cannot do without --------------------------------------------------


def work(case):
    c, io = case, 2 if case["dtype"] == "bf16" else 4
    B, L = c["B"], c["L"]
    if c["op"] == "conv":
        C, K = c["C"], c["K"]
        w, st = C * (K + 1) * 4, B * (K - 1) * C * io
        if c["dir"] == "backward":  # x and dy in, dx out, the weight and its gradient
            return {"bytes": 3 * B * L * C * io + 2 * w + 3 * st * c["state"], "flops": 6 * B * L * C * K}
        return {"bytes": 2 * B * L * C * io + w + st * (1 + c["state"]), "flops": 2 * B * L * C * K}
    if c["op"] == "scan":
        H, P, G, N = c["H"], c["P"], c["G"], c["N"]
        x, dt, bc, st = B * L * H * P * io, B * L * H * io, B * L * G * N * io, B * H * N * P * 4
        if c["dir"] == "backward":  # x, dy, dt, B, C in; dx, ddt, dB, dC out
            return {"bytes": 3 * x + 2 * dt + 4 * bc + 3 * st * c["state"],
                    "flops": 12 * B * L * H * N * P}
        return {"bytes": 2 * x + dt + 2 * bc + st * (1 + c["state"]), "flops": 5 * B * L * H * N * P}
    D, rt = c["D"], 2 if c["resid"] == "bf16" else 4
    g = {"token": B * L * D * io, "sequence": B * D * 4, "channel": D * 4}.get(c["gate"], 0)
    params = 4 * D * (2 + c["scale"] + 2 * (c["kind"] == "layer"))
    if c["dir"] == "backward":  # resid, y, gate and the outputs' gradients in; as many gradients out
        return {"bytes": B * L * D * (3 * rt + 3 * io) + 2 * g + 2 * params, "flops": 40 * B * L * D}
    return {"bytes": B * L * D * (2 * rt + 2 * io) + g + params, "flops": 16 * B * L * D}
