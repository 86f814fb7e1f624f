"""The operators around the layer around the layer itself: norm, convolution of
the block's input, the projections, TTT-Linear, the output projection and the
norm with its gate, each on what the one before it returns, against its
definition in 64 bits on those values. The projections and the layer hold
features heads first, the operators around it token by token: the layer's
output is laid out anew for the output projection's product.

Bounds: the norms and the convolution as in their own tests (96 and 32 half steps of
fp32 at the terms' magnitudes besides the output's rounding), the projections
and the layer by the bf16 bar of their parity tests, 2e-2 of a head's largest
value.
"""
import pytest
import torch

import oracle
from tests import block_ref as R
from tests import parity as P
from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu
BF, EPS = torch.bfloat16, 1e-6


@pytest.mark.parametrize("B,L,H", [(2, 70, 2), (1, 16, 3)])
def test_a_block_around_ttt_linear(B, L, H):
    g = torch.Generator().manual_seed(B)
    r = lambda *s: torch.randn(s, generator=g)
    D, K = 64 * H, 4
    resid, y = r(B, L, D).to(BF).cuda(), r(B, L, D).to(BF).cuda()
    post, pre, gate = (1 + 0.1 * r(D)).cuda(), (1 + 0.1 * r(D)).cuda(), r(B, L, D).to(BF).cuda()
    w, b, theta = (r(D, K) * K ** -0.5).cuda(), (0.1 * r(D)).cuda(), (r(3, D, D) * D ** -0.5).to(BF).cuda()
    w_out = (r(D, D) * D ** -0.5).to(BF).cuda()
    eta = torch.full((B, H, L), 1 / 64, device="cuda")
    W0, b0, gam, bet = (0.02 * r(H, 64, 64)).cuda(), torch.zeros(H, 64).cuda(), torch.ones(H, 64).cuda(), torch.zeros(H, 64).cuda()

    norm = lambda *a, **k: ttt.ttt_block_norm(*a, post, pre, eps=EPS, **k)
    ref_norm = lambda a, y, gate=None: R.block_norm(R.t64(a), R.t64(y), R.t64(post), R.t64(pre), R.t64(gate), None, None,
                                                    None, "rms", "none" if gate is None else "sigmoid", EPS, None)
    r1, x = norm(resid, y)
    for got, want, name in zip((r1, x), ref_norm(resid, y), ("resid", "x")):
        R.check(got, want, name, 96)
    c, _ = ttt.ttt_conv_forward(x, w, b)
    a = lambda t: R.t64(t).abs()
    R.check(c, R.conv(R.t64(x), R.t64(w), R.t64(b), None, "silu", None)[0], "conv", 32,
            R.conv(a(x), a(w), a(b), None, "none", None)[0])
    q, k, v = ttt.ttt_qkv_project(c, theta, H)
    for got, want in zip((q, k, v), oracle.qkv_project(P.to_np(c), P.to_np(theta), H)):
        assert P.max_rel(P.to_np(got), want, B * H) < 2e-2
    o, W, bo = ttt.ttt_linear_forward(q, k, v, eta, W0, b0, gam, bet)
    want = oracle.linear_forward(*(P.to_np(t) for t in (q, k, v, eta, W0, b0, gam, bet)), EPS)
    for got, ref in zip((o, W, bo), want):
        assert P.max_rel(P.to_np(got), ref, B * H) < 2e-2
    out = o.transpose(1, 2).reshape(B, L, D) @ w_out
    r2, x2 = norm(r1, out, gate=gate, gate_act="sigmoid")
    for got, want, name in zip((r2, x2), ref_norm(r1, out, gate), ("resid", "x")):
        R.check(got, want, name, 96)
    # the convolution's next token goes on from its last rows
    again = ttt.ttt_conv_step(x[:, 0], w, x[:, L - K + 1:].clone(), b)
    longer, _ = ttt.ttt_conv_forward(torch.cat([x, x[:, :1]], 1), w, b)
    assert torch.equal(again, longer[:, -1])
