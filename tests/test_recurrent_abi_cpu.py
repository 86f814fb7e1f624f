"""Host validation of the gated linear recurrence and the 8-bit integer
products: bad arguments are refused before any HIP call, and calls over nothing
need no pointers. No GPU: the pointers below are never dereferenced, and every
call here ends at the host's checks."""
import ctypes

import pytest

from test_sequence_layer_ttt_amd import _lib, ttt

MB = 1 << 20
PTR = [0x10000000 + i * 64 * MB for i in range(64)]  # far apart, 16-byte aligned
SHAPE, NULL, DTYPE, ALIGN, ALIAS = (_lib.TTT_E_SHAPE, _lib.TTT_E_NULL, _lib.TTT_E_DTYPE, _lib.TTT_E_ALIGN,
                                    _lib.TTT_E_ALIAS)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def s(*v):
    return (ctypes.c_int64 * len(v))(*v)


def call(lib, fn, **over):
    spec = ALL[fn]
    unknown = set(over) - {k for k, _ in spec}
    assert not unknown, unknown
    return getattr(lib, fn)(*[over.get(k, v) for k, v in spec], None)


def msg(lib):
    return lib.ttt_last_error().decode()


LRU = [("B", 2), ("L", 200), ("D", 64), ("io", 1), ("x", PTR[0]), ("xs", None), ("r", PTR[1]), ("rs", None), ("i", PTR[2]),
       ("is", None), ("rate", PTR[3]), ("state", PTR[4]), ("lens", PTR[5])]
ALL = {
    "ttt_lru_forward": LRU + [("y", PTR[6]), ("ys", None), ("so", PTR[7]), ("ws", PTR[8]), ("bytes", 1 << 30)],
    "ttt_lru_step": [("B", 2), ("D", 64), ("io", 1), ("x", PTR[0]), ("xs", None), ("r", PTR[1]), ("rs", None),
                     ("i", PTR[2]), ("is", None), ("rate", PTR[3]), ("state", PTR[4]), ("y", PTR[6])],
    "ttt_lru_backward": LRU + [("dy", PTR[6]), ("dys", None), ("dso", PTR[7]), ("dx", PTR[8]), ("dxs", None),
                               ("dr", PTR[9]), ("drs", None), ("di", PTR[10]), ("dis", None), ("drate", PTR[11]),
                               ("dstate", PTR[12]), ("ws", PTR[13]), ("bytes", 1 << 30)],
    "ttt_i8_quantize": [("M", 4), ("K", 64), ("io", 1), ("x", PTR[0]), ("xs", None), ("q", PTR[1]), ("qs", None),
                        ("scale", PTR[2])],
    "ttt_i8_project": [("M", 4), ("K", 64), ("N", 32), ("io", 1), ("x", PTR[0]), ("xs", None), ("x_scale", PTR[1]),
                       ("w", PTR[2]), ("ws", None), ("w_scale", PTR[3]), ("bias", PTR[4]), ("y", PTR[5]), ("ys", None),
                       ("work", None), ("bytes", 0)],
    "ttt_i8_linear": [("M", 4), ("K", 64), ("N", 32), ("io", 1), ("x", PTR[0]), ("xs", None), ("w", PTR[2]), ("ws", None),
                      ("w_scale", PTR[3]), ("bias", PTR[4]), ("y", PTR[5]), ("ys", None), ("work", PTR[6]),
                      ("bytes", 1 << 30)],
    "ttt_qkv_project_i8": [("B", 2), ("L", 8), ("dm", 64), ("H", 2), ("d", 64), ("x", PTR[0]), ("theta", PTR[1]),
                           ("theta_scale", PTR[2]), ("XQ", PTR[3]), ("XK", PTR[4]), ("XV", PTR[5]), ("work", PTR[6]),
                           ("bytes", 1 << 30)],
}
BAD = [
    *[(f, k, v) for f in ("ttt_lru_forward", "ttt_lru_backward")
      for k, v in (("B", -1), ("L", -1), ("L", (1 << 30) + 1), ("L", 1 << 28), ("D", 0), ("D", -1), ("D", (1 << 20) + 1),
                   ("B", 65536))],
    *[("ttt_lru_step", k, v) for k, v in (("B", -1), ("D", 0), ("D", (1 << 20) + 1), ("B", 1 << 26))],
    *[(f, k, v) for f in ("ttt_i8_quantize", "ttt_i8_project", "ttt_i8_linear")
      for k, v in (("M", -1), ("M", (1 << 24) + 1), ("K", 0), ("K", -1), ("K", 65537))],
    *[(f, k, v) for f in ("ttt_i8_project", "ttt_i8_linear") for k, v in (("N", -1), ("N", (1 << 24) + 1))],
    *[("ttt_qkv_project_i8", k, v) for k, v in (("B", -1), ("L", -1), ("H", -1), ("d", 32), ("dm", 0), ("dm", 65537),
                                               ("B", 1 << 22), ("H", 1 << 20))],
]


@pytest.mark.parametrize("fn,key,value", BAD)
def test_refuses_arguments_out_of_range(lib, fn, key, value):
    assert call(lib, fn, **{key: value}) == SHAPE
    assert msg(lib)


def test_refuses_grids_that_32_bits_do_not_count(lib):
    assert call(lib, "ttt_lru_forward", B=1 << 15, L=64 << 7) == SHAPE
    assert "ceil(L/64)" in msg(lib)
    assert call(lib, "ttt_i8_project", M=1 << 24, N=1024) == SHAPE
    assert "ceil(M/64)" in msg(lib)


@pytest.mark.parametrize("fn", [f for f in ALL if "io" in dict(ALL[f])])
def test_refuses_types(lib, fn):
    assert call(lib, fn, io=7) == DTYPE


REQUIRED = {"ttt_lru_forward": ["x", "r", "y", "ws"], "ttt_lru_step": ["x", "r", "state", "y"],
            "ttt_lru_backward": ["x", "r", "dy", "dx", "dr", "di", "drate", "dstate", "ws"],
            "ttt_i8_quantize": ["x", "scale"], "ttt_i8_project": ["x_scale", "w_scale", "y"],
            "ttt_i8_linear": ["x", "w_scale", "y", "work"], "ttt_qkv_project_i8": ["x", "theta_scale", "XQ", "XK", "XV", "work"]}


@pytest.mark.parametrize("fn,key", [(f, k) for f, v in REQUIRED.items() for k in v])
def test_refuses_null_and_misaligned(lib, fn, key):
    assert call(lib, fn, **{key: None}) == NULL, key
    assert call(lib, fn, **{key: dict(ALL[fn])[key] + 1}) == ALIGN, key


def test_rows_of_bytes_have_any_address(lib):
    for fn, key in (("ttt_i8_quantize", "q"), ("ttt_i8_project", "x"), ("ttt_i8_project", "w"), ("ttt_i8_linear", "w"),
                    ("ttt_qkv_project_i8", "theta")):
        assert call(lib, fn, **{key: None}) == NULL, key
    assert call(lib, "ttt_i8_project", M=0, x=PTR[0] + 1) == _lib.TTT_OK


def test_refuses_gradients_without_their_operand(lib):
    for k in ("i", "rate", "state"):
        assert call(lib, "ttt_lru_backward", **{k: None}) == NULL


OUTPUTS = {"ttt_lru_forward": ["y", "so", "ws"], "ttt_lru_step": ["state", "y"],
           "ttt_lru_backward": ["dx", "dr", "di", "drate", "dstate", "ws"], "ttt_i8_quantize": ["q", "scale"],
           "ttt_i8_project": ["y"], "ttt_i8_linear": ["y", "work"], "ttt_qkv_project_i8": ["XQ", "XK", "XV", "work"]}


@pytest.mark.parametrize("fn,key", [(f, k) for f, v in OUTPUTS.items() for k in v])
def test_refuses_outputs_over_inputs_and_each_other(lib, fn, key):
    spec = dict(ALL[fn])
    assert call(lib, fn, **{key: spec["x"]}) == ALIAS
    assert "overlaps" in msg(lib)
    for other in OUTPUTS[fn]:
        if other != key:
            assert call(lib, fn, **{key: spec[other]}) == ALIAS
    if key == "so":  # the state may be replaced exactly where it stands, not beside it
        assert call(lib, fn, so=spec["state"] + 16) == ALIAS


def test_refuses_strides(lib):
    assert call(lib, "ttt_lru_forward", xs=s(-12800, 64)) == SHAPE
    assert "negative stride" in msg(lib)
    assert call(lib, "ttt_lru_forward", ys=s(12800, 32)) == SHAPE
    assert "share addresses" in msg(lib)
    assert call(lib, "ttt_lru_backward", dis=s(0, 64)) == SHAPE
    assert call(lib, "ttt_lru_forward", rs=s(1 << 62, 64)) == SHAPE
    assert "overflow" in msg(lib)
    assert call(lib, "ttt_i8_project", ys=s(16)) == SHAPE
    assert call(lib, "ttt_i8_quantize", qs=s(63)) == SHAPE
    assert call(lib, "ttt_i8_project", ws=s(-64)) == SHAPE
    # columns of one buffer overlap where they share columns
    base, row = PTR[30], 192
    kw = dict(dx=base, dxs=s(200 * row, row), dr=base + 2 * 32, drs=s(200 * row, row))
    assert call(lib, "ttt_lru_backward", **kw) == ALIAS


QUERIES = [("ttt_lru_forward", ttt.ttt_lru_forward_workspace, (2, 200, 64), "bytes"),
           ("ttt_lru_backward", ttt.ttt_lru_backward_workspace, (2, 200, 64), "bytes")]


@pytest.mark.parametrize("fn,query,args,key", QUERIES, ids=lambda v: getattr(v, "__name__", None))
def test_workspaces(lib, fn, query, args, key):
    n = query(*args)
    assert n > 0
    assert call(lib, fn, **{key: n - 1}) == SHAPE
    assert "workspace" in msg(lib)
    for i in range(len(args)):
        with pytest.raises(ValueError, match="too large"):
            query(*args[:i], args[i] + 2**32, *args[i + 1:])
        with pytest.raises(ttt.TTTError):
            query(*args[:i], -1, *args[i + 1:])
    assert getattr(lib, query.__name__)(*args, None) == NULL


def _need(lib, fn, *args):
    n = ctypes.c_size_t(0)
    assert getattr(lib, fn)(*args, ctypes.byref(n)) == _lib.TTT_OK
    return n.value


@pytest.mark.parametrize("fn,query,at", [("ttt_i8_linear", (4, 64, 32, PTR[2], None), {}),
                                         ("ttt_i8_linear", (100, 64, 32, PTR[2] + 1, None), dict(M=100, w=PTR[2] + 1)),
                                         ("ttt_qkv_project_i8", (16, 64, 384, PTR[1], None), {}),
                                         ("ttt_qkv_project_i8", (100, 72, 384, PTR[1], None), dict(L=50, dm=72))])
def test_workspaces_of_products_of_features(lib, fn, query, at):
    """The quantised rows and, with more than 64 of them, a weight whose rows are no whole chunks."""
    n = _need(lib, "ttt_i8_linear_workspace", *query)
    M, K, N, w, _ = query
    pad = -(-K // 128) * 128
    assert n == M * pad + -(-M // 4) * 16 + (N * pad if M > 64 and (K % 16 or w % 16) else 0)
    assert call(lib, fn, **at, bytes=n - 1) == SHAPE
    assert "workspace" in msg(lib)
    assert call(lib, fn, **at, work=PTR[6] + 8) == ALIGN


def test_workspaces_of_products_of_rows(lib):
    q = lambda M, K, N, x=PTR[0], xs=None, w=PTR[2], ws=None: _need(lib, "ttt_i8_project_workspace", M, K, N, x, xs, w, ws)
    assert q(100, 64, 32) == 0 and q(64, 65, 32) == 0 and q(0, 65, 32) == 0 and q(100, 65, 0) == 0
    assert q(100, 65, 32) == (100 + 32) * 128
    assert q(100, 64, 32, x=PTR[0] + 8) == 100 * 128 and q(100, 64, 32, w=PTR[2] + 1) == 32 * 128
    assert q(100, 64, 32, xs=s(72)) == 100 * 128 and q(100, 64, 32, ws=s(1 << 23)) == 32 * 128
    kw = dict(M=100, K=65)
    assert call(lib, "ttt_i8_project", **kw) == SHAPE and "workspace" in msg(lib)
    assert call(lib, "ttt_i8_project", **kw, work=PTR[9], bytes=132 * 128 - 1) == SHAPE
    assert call(lib, "ttt_i8_project", **kw, work=None, bytes=1 << 20) == NULL
    assert call(lib, "ttt_i8_project", **kw, work=PTR[9] + 8, bytes=1 << 20) == ALIGN
    assert call(lib, "ttt_i8_project", **kw, work=PTR[0], bytes=1 << 20) == ALIAS
    for f, args in (("ttt_i8_project_workspace", (4, 64, 32, None, None, None, None)), ("ttt_i8_linear_workspace", (4, 64, 32, None, None))):
        assert getattr(lib, f)(*args, None) == NULL
        n = ctypes.c_size_t(0)
        for i in range(3):
            assert getattr(lib, f)(*args[:i], -1, *args[i + 1:], ctypes.byref(n)) == SHAPE


def test_workspace_queries_in_python():
    import torch
    w = torch.zeros(32, 64, dtype=torch.int8)
    assert ttt.ttt_i8_linear_workspace(100, w) == 100 * 128 + 400
    assert ttt.ttt_i8_linear_workspace(100, w[:, 1:]) == 132 * 128 + 400
    assert ttt.ttt_i8_project_workspace(100, w[:, 1:], w[:, 1:]) == 132 * 128
    assert ttt.ttt_i8_project_workspace(64, w[:, 1:], w[:, 1:]) == 0
    for fn, args in ((ttt.ttt_i8_linear_workspace, (w,)), (ttt.ttt_i8_project_workspace, (w, w))):
        with pytest.raises(ValueError, match="too large"):
            fn(2**32, *args)
        with pytest.raises(ttt.TTTError):
            fn(-1, *args)
        with pytest.raises(TypeError):
            fn(1, *(t.float() for t in args))


def test_empty_calls_launch_nothing(lib):
    assert call(lib, "ttt_lru_forward", B=0) == _lib.TTT_OK
    assert call(lib, "ttt_lru_forward", L=0, so=None, x=None, r=None, y=None, i=None, ws=None) == _lib.TTT_OK
    assert call(lib, "ttt_lru_step", B=0) == _lib.TTT_OK
    assert call(lib, "ttt_i8_quantize", M=0, x=None, q=None, scale=None) == _lib.TTT_OK
    assert call(lib, "ttt_i8_project", M=0, x=None, x_scale=None, y=None) == _lib.TTT_OK
    assert call(lib, "ttt_i8_project", N=0, w=None, w_scale=None, y=None, bias=None) == _lib.TTT_OK
    assert call(lib, "ttt_i8_linear", M=0, x=None, y=None, work=None, bytes=0) == _lib.TTT_OK
    assert call(lib, "ttt_qkv_project_i8", H=0, theta=None, theta_scale=None, XQ=None, XK=None, XV=None) == _lib.TTT_OK
    assert call(lib, "ttt_qkv_project_i8", L=0, x=None, XQ=None, XK=None, XV=None, work=None, bytes=0) == _lib.TTT_OK


@pytest.mark.parametrize("query", [ttt.ttt_lru_forward_workspace, ttt.ttt_lru_backward_workspace])
def test_grids_are_counted_in_32_bits(query):
    query(1, 1 << 26, 1024)
    query(65535, 64, 1 << 20)  # one tile a sequence: a grid of two dimensions
    for sizes in ((1, 1 << 26, 2048), (1, 1 << 27, 1024), (65535, 65, 1 << 15)):
        with pytest.raises(ttt.TTTError, match=r"ceil\(D/128\)"):
            query(*sizes)
