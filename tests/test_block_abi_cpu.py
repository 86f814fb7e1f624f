"""Host validation of the operators around the layer: bad arguments are
refused before any HIP call, and calls over nothing need no pointers. No GPU:
the pointers below are never dereferenced, and every call here ends at the
host's checks."""
import ctypes

import pytest

from test_sequence_layer_ttt_amd import _lib

MB = 1 << 20
PTR = [0x10000000 + i * 64 * MB for i in range(64)]  # far apart, 16-byte aligned
SHAPE, NULL, DTYPE, ALIGN, ALIAS = (_lib.TTT_E_SHAPE, _lib.TTT_E_NULL, _lib.TTT_E_DTYPE, _lib.TTT_E_ALIGN,
                                    _lib.TTT_E_ALIAS)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def s(*v):
    return (ctypes.c_int64 * len(v))(*v)


def call(lib, fn, spec, **over):
    """spec: (name, value) in the ABI's order; `over` replaces values."""
    unknown = set(over) - {k for k, _ in spec}
    assert not unknown, unknown
    return getattr(lib, fn)(*[over.get(k, v) for k, v in spec], None)


def msg(lib):
    return lib.ttt_last_error().decode()


CONV = [("B", 2), ("L", 8), ("C", 16), ("K", 4), ("io", 1), ("act", 2), ("x", PTR[0]), ("xs", None), ("w", PTR[1]),
        ("bias", PTR[2]), ("state", PTR[3]), ("lens", PTR[4])]
CONV_F = CONV + [("y", PTR[5]), ("ys", None), ("so", PTR[6])]
CONV_S = [("B", 2), ("C", 16), ("K", 4), ("io", 1), ("act", 2), ("x", PTR[0]), ("xs", None), ("w", PTR[1]),
          ("bias", PTR[2]), ("state", PTR[3]), ("y", PTR[5])]
CONV_B = CONV + [("dy", PTR[5]), ("dys", None), ("dso", PTR[6]), ("dx", PTR[7]), ("dxs", None), ("dw", PTR[8]),
                 ("dbias", PTR[9]), ("dstate", PTR[10]), ("ws", PTR[11]), ("bytes", 1 << 30)]
SSM = [("B", 2), ("L", 8), ("H", 4), ("P", 64), ("G", 2), ("N", 32), ("io", 1), ("x", PTR[0]), ("xs", None),
       ("dt", PTR[1]), ("dts", None), ("A", PTR[2]), ("Bm", PTR[3]), ("bs", None), ("Cm", PTR[4]), ("cs", None),
       ("D", PTR[5]), ("dtb", PTR[6]), ("state", PTR[7]), ("lens", PTR[8])]
SSM_F = SSM + [("y", PTR[9]), ("ys", None), ("so", PTR[10]), ("ws", PTR[11]), ("bytes", 1 << 30)]
SSM_S = [("B", 2), ("H", 4), ("P", 64), ("G", 2), ("N", 32), ("io", 1), ("x", PTR[0]), ("xs", None), ("dt", PTR[1]),
         ("dts", None), ("A", PTR[2]), ("Bm", PTR[3]), ("bs", None), ("Cm", PTR[4]), ("cs", None), ("D", PTR[5]),
         ("dtb", PTR[6]), ("state", PTR[7]), ("y", PTR[9])]
SSM_B = SSM + [("dy", PTR[9]), ("dys", None), ("dso", PTR[10]), ("dx", PTR[11]), ("dxs", None), ("ddt", PTR[12]),
               ("ddts", None), ("dA", PTR[13]), ("dB", PTR[14]), ("dbs", None), ("dC", PTR[15]), ("dcs", None),
               ("dD", PTR[16]), ("ddtb", PTR[17]), ("dstate", PTR[18]), ("ws", PTR[19]), ("bytes", 1 << 30)]
NORM = [("B", 2), ("L", 8), ("D", 64), ("io", 1), ("rio", 0), ("layer", 0), ("shape", 3), ("act", 1), ("eps", 1e-6),
        ("resid", PTR[0]), ("rs", None), ("y", PTR[1]), ("ys", None), ("gate", PTR[2]), ("gs", None), ("pg", PTR[3]),
        ("pb", PTR[4]), ("qg", PTR[5]), ("qb", PTR[6]), ("scale", PTR[7]), ("lens", PTR[8])]
NORM_F = NORM + [("ro", PTR[9]), ("xo", PTR[10])]
NORM_B = NORM + [("dro", PTR[9]), ("dx", PTR[10]), ("dresid", PTR[11]), ("dy", PTR[12]), ("dgate", PTR[13]),
                 ("dpg", PTR[14]), ("dpb", PTR[15]), ("dqg", PTR[16]), ("dqb", PTR[17]), ("dscale", PTR[18]),
                 ("ws", PTR[19]), ("bytes", 1 << 30)]
ALL = {"ttt_conv_forward": CONV_F, "ttt_conv_step": CONV_S, "ttt_conv_backward": CONV_B, "ttt_ssm_forward": SSM_F,
       "ttt_ssm_step": SSM_S, "ttt_ssm_backward": SSM_B, "ttt_block_norm": NORM_F, "ttt_block_norm_backward": NORM_B}


@pytest.mark.parametrize("fn", list(ALL))
def test_refuses_sizes_and_types(lib, fn):
    spec = ALL[fn]
    assert call(lib, fn, spec, B=-1) == SHAPE
    assert "negative" in msg(lib)
    assert call(lib, fn, spec, io=7) == DTYPE
    if "L" in dict(spec):
        assert call(lib, fn, spec, L=(1 << 30) + 1, B=1) == SHAPE


BAD = [
    *[(f, k, v) for f in ("ttt_conv_forward", "ttt_conv_step", "ttt_conv_backward")
      for k, v in (("K", 1), ("K", 5), ("C", -1), ("C", (1 << 20) + 1), ("act", 1), ("act", 3))],
    *[(f, k, v) for f in ("ttt_conv_forward", "ttt_conv_backward") for k, v in (("B", 65536),)],
    ("ttt_conv_step", "B", 1 << 30),
    *[(f, k, v) for f in ("ttt_ssm_forward", "ttt_ssm_step", "ttt_ssm_backward")
      for k, v in (("P", 0), ("P", 129), ("N", 0), ("N", 129), ("G", 3), ("G", 0), ("H", 0), ("B", 1 << 21))],
    *[(f, "L", 1 << 26) for f in ("ttt_ssm_forward", "ttt_ssm_backward")],
    *[(f, k, v) for f in ("ttt_block_norm", "ttt_block_norm_backward")
      for k, v in (("D", 0), ("D", 8193), ("layer", 2), ("act", 4), ("act", -1), ("shape", 4), ("eps", 0.0),
                   ("eps", float("nan")), ("eps", 1e-40), ("L", 1 << 30))],
]


@pytest.mark.parametrize("fn,key,value", BAD)
def test_refuses_arguments_out_of_range(lib, fn, key, value):
    assert call(lib, fn, ALL[fn], **{key: value}) == SHAPE
    assert msg(lib)


def test_refuses_a_residual_of_another_type(lib):
    for fn in ("ttt_block_norm", "ttt_block_norm_backward"):
        assert call(lib, fn, ALL[fn], io=0, rio=1) == DTYPE
    assert call(lib, "ttt_block_norm", NORM_F, shape=2, B=65536, L=1) == SHAPE


REQUIRED = {"ttt_conv_forward": ["x", "w", "y"], "ttt_conv_step": ["x", "w", "state", "y"],
            "ttt_conv_backward": ["x", "w", "dy", "dx", "dw", "dbias", "dstate", "ws"],
            "ttt_ssm_forward": ["x", "dt", "A", "Bm", "Cm", "y"],
            "ttt_ssm_step": ["x", "dt", "A", "Bm", "Cm", "state", "y"],
            "ttt_ssm_backward": ["x", "dt", "A", "Bm", "Cm", "dy", "dx", "ddt", "dA", "dB", "dC", "dD", "ddtb",
                                 "dstate", "ws"],
            "ttt_block_norm": ["resid", "y", "gate", "ro", "xo"],
            "ttt_block_norm_backward": ["resid", "y", "gate", "dro", "dx", "dresid", "dy", "dgate", "ws"]}


@pytest.mark.parametrize("fn,key", [(f, k) for f, v in REQUIRED.items() for k in v])
def test_refuses_null_and_misaligned(lib, fn, key):
    assert call(lib, fn, ALL[fn], **{key: None}) == NULL, key
    assert call(lib, fn, ALL[fn], **{key: dict(ALL[fn])[key] + 1}) == ALIGN, key


def test_refuses_gradients_without_their_operand(lib):
    """dbias without bias, dstate without state, dD without D and the like."""
    assert call(lib, "ttt_conv_backward", CONV_B, bias=None) == NULL
    assert call(lib, "ttt_conv_backward", CONV_B, state=None) == NULL
    for k in ("D", "dtb", "state"):
        assert call(lib, "ttt_ssm_backward", SSM_B, **{k: None}) == NULL


OUTPUTS = {"ttt_conv_forward": ["y", "so"], "ttt_conv_step": ["state", "y"],
           "ttt_conv_backward": ["dx", "dw", "dbias", "dstate", "ws"], "ttt_ssm_forward": ["y", "so"],
           "ttt_ssm_step": ["state", "y"],
           "ttt_ssm_backward": ["dx", "ddt", "dA", "dB", "dC", "dD", "ddtb", "dstate", "ws"],
           "ttt_block_norm": ["ro", "xo"],
           "ttt_block_norm_backward": ["dresid", "dy", "dgate", "dpg", "dpb", "dqg", "dqb", "dscale", "ws"]}


@pytest.mark.parametrize("fn,key", [(f, k) for f, v in OUTPUTS.items() for k in v])
def test_refuses_outputs_over_inputs_and_each_other(lib, fn, key):
    spec = dict(ALL[fn])
    first_in = "resid" if "resid" in spec else "x"
    assert call(lib, fn, ALL[fn], **{key: spec[first_in]}) == ALIAS
    assert "overlaps" in msg(lib)
    for other in OUTPUTS[fn]:
        if other != key:
            assert call(lib, fn, ALL[fn], **{key: spec[other]}) == ALIAS
    # the state may be replaced exactly where it stands, not beside it
    if key == "so":
        assert call(lib, fn, ALL[fn], so=spec["state"] + 16) == ALIAS


def test_refuses_strides(lib):
    assert call(lib, "ttt_conv_forward", CONV_F, xs=s(-128, 16)) == SHAPE
    assert "negative stride" in msg(lib)
    assert call(lib, "ttt_conv_forward", CONV_F, ys=s(128, 8)) == SHAPE  # rows of 16 that overlap
    assert "share addresses" in msg(lib)
    assert call(lib, "ttt_conv_forward", CONV_F, ys=s(0, 16)) == SHAPE
    assert call(lib, "ttt_ssm_forward", SSM_F, ys=s(2048, 256, 32)) == SHAPE
    assert call(lib, "ttt_ssm_forward", SSM_F, xs=s(1 << 62, 256, 64)) == SHAPE
    assert "overflow" in msg(lib)
    # columns of one buffer overlap where they share columns or rows differ
    base, row = PTR[30], 64
    kw = dict(x=base, xs=s(8 * row, row), y=base + 2 * 8, ys=s(8 * row, row))
    assert call(lib, "ttt_conv_forward", CONV_F, **kw) == ALIAS
    kw = dict(x=base, xs=s(8 * row, row), y=base + 2 * 16, ys=s(8 * (row + 16), row + 16))
    assert call(lib, "ttt_conv_forward", CONV_F, **kw) == ALIAS
    kw = dict(x=base, xs=s(8 * row, row), y=base + 2 * 56, ys=s(8 * row, row))  # reaches into the next row
    assert call(lib, "ttt_conv_forward", CONV_F, **kw) == ALIAS


@pytest.mark.parametrize("fn,query,args", [
    ("ttt_conv_backward", "ttt_conv_backward_workspace", (2, 8, 16, 4)),
    ("ttt_ssm_backward", "ttt_ssm_backward_workspace", (2, 8, 4, 64, 2, 32)),
    ("ttt_block_norm_backward", "ttt_block_norm_backward_workspace", (2, 8, 64, 3))])
def test_workspaces(lib, fn, query, args):
    n = ctypes.c_size_t(0)
    assert getattr(lib, query)(*args, ctypes.byref(n)) == _lib.TTT_OK and n.value > 0
    assert call(lib, fn, ALL[fn], bytes=n.value - 1) == SHAPE
    assert "workspace" in msg(lib)
    assert getattr(lib, query)(*args, None) == NULL


def test_workspace_of_a_segmented_prompt(lib):
    n = ctypes.c_size_t(0)
    assert lib.ttt_ssm_forward_workspace(1, 8192, 4, 64, 1, 64, ctypes.byref(n)) == _lib.TTT_OK and n.value > 0
    assert call(lib, "ttt_ssm_forward", SSM_F, B=1, L=8192, G=1, N=64, bytes=n.value - 1) == SHAPE


def test_the_scan_refuses_grids_that_32_bits_do_not_count(lib):
    """B*H*ceil(L/64) has to stay below 2^22."""
    n = ctypes.c_size_t(0)
    for q in (lib.ttt_ssm_forward_workspace, lib.ttt_ssm_backward_workspace):
        assert q(1, 64 * ((1 << 22) - 1), 1, 1, 1, 1, ctypes.byref(n)) == _lib.TTT_OK
        assert q(1, 64 << 22, 1, 1, 1, 1, ctypes.byref(n)) == SHAPE
        assert q(1 << 11, 64, 1 << 11, 1, 1, 1, ctypes.byref(n)) == SHAPE


def test_empty_batches_launch_nothing(lib):
    z = dict(B=0)
    assert call(lib, "ttt_conv_forward", CONV_F, **z) == _lib.TTT_OK
    assert call(lib, "ttt_conv_step", CONV_S, **z) == _lib.TTT_OK
    assert call(lib, "ttt_ssm_forward", SSM_F, **z) == _lib.TTT_OK
    assert call(lib, "ttt_ssm_step", SSM_S, **z) == _lib.TTT_OK
    assert call(lib, "ttt_block_norm", NORM_F, **z) == _lib.TTT_OK
    assert call(lib, "ttt_conv_forward", CONV_F, L=0, so=None, x=None, y=None) == _lib.TTT_OK
    assert call(lib, "ttt_block_norm", NORM_F, L=0) == _lib.TTT_OK


def test_the_binding_declares_every_argument():
    """ctypes passes what argtypes name: as many as the header declares."""
    import re
    header = open(_lib.HEADER).read()
    lib = _lib.load()
    for name in _lib.header_functions():
        args = re.search(r"\b" + name + r"\s*\(([^;]*)\);", header).group(1).split(",")
        types = getattr(lib, name).argtypes
        if types is not None:
            assert len(types) == len([a for a in args if a.strip() != "void"]), name
