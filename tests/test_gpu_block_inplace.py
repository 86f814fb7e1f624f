"""What the operators around the layer write into a tensor of the caller's, a
state in place or an output that is given, counts as a change of it: torch's
autograd refuses to go back through what it had saved of the tensor before."""
import pytest
import torch

from test_sequence_layer_ttt_amd import ttt

pytestmark = pytest.mark.gpu


def _calls(dt=torch.bfloat16):
    """name -> (call, tensors that it writes, tensors that it reads)"""
    r = lambda *s: torch.randn(*s, device="cuda")
    B, L, C, K, H, P, N, D = 2, 5, 16, 4, 2, 8, 4, 32
    x, w, cs, cy, so = r(B, L, C).to(dt), r(C, K), r(B, K - 1, C).to(dt), r(B, L, C).to(dt), r(B, K - 1, C).to(dt)
    out = {"conv_forward": (lambda: ttt.ttt_conv_forward(x, w, state=cs, y=cy, state_out=so), [cy, so], [x, w, cs]),
           "conv_in_place": (lambda: ttt.ttt_conv_forward(x, w, state=cs, state_out=cs), [cs], [x, w])}
    ty = r(B, C).to(dt)
    out["conv_step"] = (lambda: ttt.ttt_conv_step(x[:, 0], w, cs), [cs], [x, w])
    out["conv_step_y"] = (lambda: ttt.ttt_conv_step(x[:, 0], w, cs, y=ty), [cs, ty], [x, w])
    cg = {"dx": r(B, L, C).to(dt), "dweight": r(C, K), "dstate": r(B, K - 1, C).to(dt)}
    out["conv_backward"] = (lambda: ttt.ttt_conv_backward(x, w, x, state=cs, grads=cg), list(cg.values()), [x, w, cs])
    sx, sdt, A, Bm, Cm = r(B, L, H, P).to(dt), r(B, L, H).to(dt), -r(H).abs(), r(B, L, 1, N).to(dt), r(B, L, 1, N).to(dt)
    st, sy, ss, sty = r(B, H, N, P), r(B, L, H, P).to(dt), r(B, H, N, P), r(B, H, P).to(dt)
    out["ssm_forward"] = (lambda: ttt.ttt_ssm_forward(sx, sdt, A, Bm, Cm, state=st, y=sy, state_out=ss), [sy, ss],
                          [sx, sdt, A, Bm, Cm, st])
    out["ssm_in_place"] = (lambda: ttt.ttt_ssm_forward(sx, sdt, A, Bm, Cm, state=st, state_out=st), [st], [sx, A])
    out["ssm_step"] = (lambda: ttt.ttt_ssm_step(sx[:, 0], sdt[:, 0], A, Bm[:, 0], Cm[:, 0], st, y=sty), [st, sty], [sx, A])
    sg = {"dx": r(B, L, H, P).to(dt), "ddt": r(B, L, H).to(dt), "dA": r(H), "dB": r(B, L, 1, N).to(dt),
          "dC": r(B, L, 1, N).to(dt), "dstate": r(B, H, N, P)}
    out["ssm_backward"] = (lambda: ttt.ttt_ssm_backward(sx, sdt, A, Bm, Cm, sx, state=st, grads=sg), list(sg.values()),
                           [sx, A, st])
    res, y, ro, xo = r(B, L, D), r(B, L, D).to(dt), r(B, L, D), r(B, L, D).to(dt)
    out["block_norm"] = (lambda: ttt.ttt_block_norm(res, y, resid_out=ro, x=xo), [ro, xo], [res, y])
    ng = {"dresid": r(B, L, D), "dy": r(B, L, D).to(dt)}
    out["block_norm_backward"] = (lambda: ttt.ttt_block_norm_backward(res, y, None, None, res, y, grads=ng),
                                  list(ng.values()), [res, y])
    return out


NAMES = ["conv_forward", "conv_in_place", "conv_step", "conv_step_y", "conv_backward", "ssm_forward", "ssm_in_place",
         "ssm_step", "ssm_backward", "block_norm", "block_norm_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_written_tensors_change_their_version(name):
    fn, writes, reads = _calls()[name]
    before = [t._version for t in writes], [t._version for t in reads]
    fn()
    assert all(t._version > v for t, v in zip(writes, before[0]))
    assert [t._version for t in reads] == before[1]


def test_autograd_refuses_a_state_that_a_step_has_changed():
    g = lambda *s: torch.randn(*s, device="cuda")
    state, w = g(2, 2, 4, 8), g(2, 2, 4, 8).requires_grad_(True)
    loss = (state * w).sum()  # saves the state for w's gradient
    ttt.ttt_ssm_step(g(2, 2, 8), g(2, 2), -g(2).abs(), g(2, 1, 4), g(2, 1, 4), state)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()


def test_tensors_of_inference_mode_are_taken():
    """They have no version."""
    with torch.inference_mode():
        calls = _calls()
        calls["ssm_step"][0]()
    for name in NAMES:
        calls[name][0]()
    torch.cuda.synchronize()
