"""Refusals of the RMS-norm, product and dropout entries (no GPU: an invalid
call returns its code before anything is enqueued), their workspace sizes, and
the plain fp64 definitions against differences and known words."""
import numpy as np
import pytest

from helpers import ensure_built
from oracle import operators as ref

ensure_built()
import cnn_convolution_conv2d_amd as c2  # noqa: E402

P, Q, R, S = 0x1000, 0x2000, 0x3000, 0x4000   # aligned addresses; nothing is dereferenced by validation
BIG = 1 << 40
TOP = 2 ** 31 - 1


def _rms(entry, **over):
    a = dict(x=P, r=Q, gamma=P, h=R, y=S, qs=P, rstd=P, dgamma=P, ws=P, bytes=BIG, M=3, C=64, ldx=64, ldr=64, ldh=64,
             ldy=64, eps=1e-5, dtype=c2.BF16)
    a.update(over)
    size = (a["M"], a["C"], a["ldx"], a["ldr"], a["ldh"], a["ldy"])
    if entry == "bwd":
        return c2.lib.conv2d_rms_norm_bwd(a["x"], a["r"], a["h"], a["gamma"], a["rstd"], a["y"], a["dgamma"], a["ws"],
                                          a["bytes"], *size, a["dtype"], None)
    if entry == "quant":
        return c2.lib.conv2d_rms_norm_quant(a["x"], a["r"], a["gamma"], a["h"], a["y"], a["qs"], a["rstd"], *size,
                                            a["eps"], a["dtype"], None)
    return c2.lib.conv2d_rms_norm(a["x"], a["r"], a["gamma"], a["h"], a["y"], a["rstd"], *size, a["eps"], a["dtype"], None)


@pytest.mark.parametrize("entry", ["fwd", "quant", "bwd"])
@pytest.mark.parametrize("over,code", [
    ({"M": 0}, c2.ERR_ARG), ({"M": -1}, c2.ERR_ARG), ({"C": 0}, c2.ERR_ARG), ({"ldx": 63}, c2.ERR_ARG),
    ({"ldr": 63}, c2.ERR_ARG), ({"ldh": 63}, c2.ERR_ARG), ({"ldy": 63}, c2.ERR_ARG), ({"ldy": -64}, c2.ERR_ARG),
    ({"dtype": 2}, c2.ERR_DTYPE), ({"x": None}, c2.ERR_NULL), ({"y": None}, c2.ERR_NULL), ({"x": P + 1}, c2.ERR_ALIGN),
    ({"r": Q + 1}, c2.ERR_ALIGN), ({"h": R + 1}, c2.ERR_ALIGN), ({"gamma": P + 2}, c2.ERR_ALIGN),
    ({"rstd": P + 2}, c2.ERR_ALIGN), ({"C": 16385, "ldx": TOP, "ldr": TOP, "ldh": TOP, "ldy": TOP}, c2.ERR_UNSUPPORTED),
], ids=str)
def test_rms_refusals(entry, over, code):
    assert _rms(entry, **over) == code
    assert c2.last_error()


@pytest.mark.parametrize("entry,over,code", [
    ("fwd", {"eps": -1e-5}, c2.ERR_ARG), ("quant", {"eps": float("nan")}, c2.ERR_ARG),
    ("fwd", {"eps": float("inf")}, c2.ERR_ARG), ("fwd", {"y": S + 1}, c2.ERR_ALIGN),
    ("fwd", {"y": R}, c2.ERR_ARG),                                     # h and y
    ("fwd", {"y": P, "ldy": 72}, c2.ERR_ARG), ("fwd", {"y": Q, "ldy": 72}, c2.ERR_ARG),
    ("fwd", {"h": P, "ldh": 72}, c2.ERR_ARG), ("quant", {"h": Q, "ldh": 72}, c2.ERR_ARG),
    ("quant", {"y": P}, c2.ERR_ARG), ("quant", {"y": Q}, c2.ERR_ARG), ("quant", {"y": R}, c2.ERR_ARG),
    ("quant", {"qs": None}, c2.ERR_NULL), ("quant", {"qs": P + 1}, c2.ERR_ALIGN),
    ("bwd", {"h": None}, c2.ERR_NULL), ("bwd", {"rstd": None}, c2.ERR_NULL), ("bwd", {"y": S + 1}, c2.ERR_ALIGN),
    ("bwd", {"dgamma": P + 1}, c2.ERR_ALIGN), ("bwd", {"ws": None}, c2.ERR_NULL), ("bwd", {"ws": P + 8}, c2.ERR_ALIGN),
    ("bwd", {"bytes": 255}, c2.ERR_ARG), ("bwd", {"y": P, "ldy": 72}, c2.ERR_ARG), ("bwd", {"y": Q, "ldy": 72}, c2.ERR_ARG),
    ("bwd", {"y": R, "ldy": 72}, c2.ERR_ARG),
], ids=str)
def test_rms_refusals_of_one_entry(entry, over, code):
    assert _rms(entry, **over) == code


def _matmul(**over):
    a = dict(x=P, w=Q, bias=P, r=R, z=0x5000, y=S, ws=P, bytes=BIG, M=8, K=64, N=32, ldx=64, ldw=64, ldr=32, ldz=32,
             ldy=32, dtype=c2.BF16, act=c2.ACT_SILU)
    a.update(over)
    return c2.lib.conv2d_matmul(a["x"], a["w"], a["bias"], a["r"], a["z"], a["y"], a["ws"], a["bytes"], a["M"], a["K"],
                                a["N"], a["ldx"], a["ldw"], a["ldr"], a["ldz"], a["ldy"], a["dtype"], a["act"], None)


LONG = (1 << 20) + 1
SPLIT = dict(M=100, K=8192, N=64, ldx=8192, ldw=8192, ldr=64, ldz=64, ldy=64)   # few tiles of long sums


@pytest.mark.parametrize("over,code", [
    ({"M": 0}, c2.ERR_ARG), ({"K": 0}, c2.ERR_ARG), ({"N": -3}, c2.ERR_ARG), ({"ldx": 63}, c2.ERR_ARG),
    ({"ldw": 63}, c2.ERR_ARG), ({"ldr": 31}, c2.ERR_ARG), ({"ldz": 31}, c2.ERR_ARG), ({"ldy": 31}, c2.ERR_ARG),
    ({"dtype": 9}, c2.ERR_DTYPE), ({"act": 4}, c2.ERR_EPILOGUE), ({"act": -1}, c2.ERR_EPILOGUE), ({"x": None}, c2.ERR_NULL),
    ({"w": None}, c2.ERR_NULL), ({"y": None}, c2.ERR_NULL), ({"x": P + 1}, c2.ERR_ALIGN), ({"w": Q + 1}, c2.ERR_ALIGN),
    ({"r": R + 1}, c2.ERR_ALIGN), ({"z": S + 1}, c2.ERR_ALIGN), ({"y": S + 1}, c2.ERR_ALIGN),
    ({"bias": P + 2}, c2.ERR_ALIGN), ({"y": P}, c2.ERR_ARG), ({"y": Q}, c2.ERR_ARG), ({"z": S}, c2.ERR_ARG),
    ({"z": P}, c2.ERR_ARG), ({"z": R}, c2.ERR_ARG), ({"y": R, "ldy": 40}, c2.ERR_ARG),
    ({"ldx": LONG}, c2.ERR_UNSUPPORTED), ({"ldw": LONG}, c2.ERR_UNSUPPORTED),
    ({"M": 1 << 30, "N": 100, "ldr": 100, "ldz": 100, "ldy": 100}, c2.ERR_UNSUPPORTED),
    ({"M": TOP, "N": 1}, c2.ERR_UNSUPPORTED),
    ({**SPLIT, "ws": None}, c2.ERR_NULL), ({**SPLIT, "bytes": 16}, c2.ERR_ARG), ({**SPLIT, "ws": P + 4}, c2.ERR_ALIGN),
], ids=str)
def test_matmul_refusals(over, code):
    assert _matmul(**over) == code
    assert c2.last_error()


def _bwd(**over):
    a = dict(dy=P, z=Q, x=R, w=S, dx=0x5000, dw=0x6000, db=0x7000, ws=P, bytes=BIG, M=8, K=64, N=32, lddy=32, ldz=32,
             ldx=64, ldw=64, lddx=64, lddw=64, dtype=c2.BF16, act=c2.ACT_SILU)
    a.update(over)
    return c2.lib.conv2d_matmul_bwd(a["dy"], a["z"], a["x"], a["w"], a["dx"], a["dw"], a["db"], a["ws"], a["bytes"], a["M"],
                                    a["K"], a["N"], a["lddy"], a["ldz"], a["ldx"], a["ldw"], a["lddx"], a["lddw"],
                                    a["dtype"], a["act"], None)


@pytest.mark.parametrize("over,code", [
    ({"M": 0}, c2.ERR_ARG), ({"K": -1}, c2.ERR_ARG), ({"N": 0}, c2.ERR_ARG), ({"lddy": 31}, c2.ERR_ARG),
    ({"ldz": 31}, c2.ERR_ARG), ({"ldx": 63}, c2.ERR_ARG), ({"ldw": 63}, c2.ERR_ARG), ({"lddx": 63}, c2.ERR_ARG),
    ({"lddw": 63}, c2.ERR_ARG), ({"dtype": 3}, c2.ERR_DTYPE), ({"act": 4}, c2.ERR_EPILOGUE), ({"dy": None}, c2.ERR_NULL),
    ({"x": None}, c2.ERR_NULL), ({"w": None}, c2.ERR_NULL), ({"z": None}, c2.ERR_NULL),
    ({"dx": None, "dw": None, "db": None}, c2.ERR_NULL), ({"dy": P + 1}, c2.ERR_ALIGN), ({"z": Q + 1}, c2.ERR_ALIGN),
    ({"dx": P + 1}, c2.ERR_ALIGN), ({"dw": P + 1}, c2.ERR_ALIGN), ({"db": P + 2}, c2.ERR_ALIGN), ({"dx": R}, c2.ERR_ARG),
    ({"dw": S}, c2.ERR_ARG), ({"dx": 0x6000}, c2.ERR_ARG), ({"lddy": LONG}, c2.ERR_UNSUPPORTED),
    ({"ldz": LONG}, c2.ERR_UNSUPPORTED), ({"ldx": LONG}, c2.ERR_UNSUPPORTED), ({"ldw": LONG}, c2.ERR_UNSUPPORTED),
    ({"M": TOP}, c2.ERR_UNSUPPORTED), ({"ws": None}, c2.ERR_NULL), ({"ws": P + 4}, c2.ERR_ALIGN), ({"bytes": 64}, c2.ERR_ARG),
], ids=str)
def test_matmul_bwd_refusals(over, code):
    assert _bwd(**over) == code
    assert c2.last_error()


@pytest.mark.parametrize("over,code", [
    ({"M": 0}, c2.ERR_ARG), ({"C": 0}, c2.ERR_ARG), ({"ldx": 63}, c2.ERR_ARG), ({"ldr": 63}, c2.ERR_ARG),
    ({"ldy": 63}, c2.ERR_ARG), ({"dtype": 5}, c2.ERR_DTYPE), ({"p": 1.0}, c2.ERR_ARG), ({"p": -0.1}, c2.ERR_ARG),
    ({"p": float("nan")}, c2.ERR_ARG), ({"x": None}, c2.ERR_NULL), ({"y": None}, c2.ERR_NULL), ({"rng": None}, c2.ERR_NULL),
    ({"x": P + 1}, c2.ERR_ALIGN), ({"r": P + 1}, c2.ERR_ALIGN), ({"y": P + 1}, c2.ERR_ALIGN), ({"rng": P + 4}, c2.ERR_ALIGN),
    ({"y": P, "ldy": 72}, c2.ERR_ARG), ({"y": Q, "ldy": 72}, c2.ERR_ARG),
], ids=str)
def test_dropout_refusals(over, code):
    a = dict(x=P, r=Q, y=S, rng=R, p=0.1, M=3, C=64, ldx=64, ldr=64, ldy=64, dtype=c2.BF16)
    a.update(over)
    assert c2.lib.conv2d_dropout(a["x"], a["r"], a["y"], a["rng"], a["p"], a["M"], a["C"], a["ldx"], a["ldr"], a["ldy"],
                                 a["dtype"], None) == code


def test_group_norm_takes_no_gelu():
    assert c2.lib.conv2d_group_norm_nhwc(P, P, P, P, P, P, P, BIG, 2, 32, 5, 7, 4, 32, 32, 1e-5, c2.BF16, c2.ACT_GELU,
                                         None) == c2.ERR_EPILOGUE


def test_the_binding_passes_every_argument():
    """Through the extension, with the code that the entry itself would return."""
    for call, code in [
            (lambda: c2.conv2d_rms_norm(P, None, None, None, S, None, 1, 4, 4, 4, 4, 3, 1e-5, c2.F32, stream=0), c2.ERR_ARG),
            (lambda: c2.conv2d_rms_norm_quant(P, None, None, None, S, None, None, 1, 4, 4, 4, 4, 4, 1e-5, c2.F32, stream=0),
             c2.ERR_NULL),
            (lambda: c2.conv2d_rms_norm_bwd(P, None, Q, None, P, S, P, None, 0, 1, 4, 4, 4, 4, 4, c2.F32, stream=0),
             c2.ERR_NULL),
            (lambda: c2.conv2d_matmul(P, Q, None, None, None, S, None, 0, 1, 1, 1, 1, 1, 1, 1, 1, c2.F32, 4, stream=0),
             c2.ERR_EPILOGUE),
            (lambda: c2.conv2d_matmul_bwd(P, Q, P, Q, None, None, None, None, 0, 1, 1, 1, 1, 1, 1, 1, 1, 1, c2.F32, 0,
                                          stream=0), c2.ERR_NULL),
            (lambda: c2.conv2d_dropout(P, None, S, Q, 1.0, 1, 1, 1, 1, 1, c2.F32, stream=0), c2.ERR_ARG)]:
        with pytest.raises(c2.Conv2dError) as e:
            call()
        assert e.value.code == code


def test_the_calls_work_without_the_extension(tmp_path, monkeypatch):
    """As the package loads where no extension is built for this Python: through ctypes, the same codes."""
    import importlib.util
    import os
    import shutil
    shutil.copy(os.path.join(os.path.dirname(c2.__file__), "__init__.py"), tmp_path)
    monkeypatch.setenv("CONV2D_LIBRARY", c2.LIB_PATH)
    spec = importlib.util.spec_from_file_location("without_extension", tmp_path / "__init__.py")
    w = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(w)
    for mod in (c2, w):
        codes = []
        for call in (lambda: mod.conv2d_rms_norm(P, None, None, None, S, None, 1, 4, 4, 4, 4, 4, -1.0, c2.F32, stream=0),
                     lambda: mod.conv2d_rms_norm_quant(P, None, None, None, P, Q, None, 1, 4, 4, 4, 4, 4, 1e-5, c2.F32, stream=0),
                     lambda: mod.conv2d_rms_norm_bwd(P, None, Q, None, P, S, P, None, 0, 1, 4, 4, 4, 4, 4, 9, stream=0),
                     lambda: mod.conv2d_matmul(P, Q, None, None, None, None, None, 0, 1, 1, 1, 1, 1, 1, 1, 1, c2.F32, 0, stream=0),
                     lambda: mod.conv2d_matmul_bwd(P, None, P, Q, S, None, None, None, 0, 1, 1, 1, 1, 1, 1, 1, 1, 1, c2.F32, 1,
                                                   stream=0),
                     lambda: mod.conv2d_dropout(P, None, S, Q, 1.5, 1, 1, 1, 1, 1, c2.F32, stream=0)):
            with pytest.raises(mod.Conv2dError) as e:
                call()
            codes.append(e.value.code)
        assert codes == [c2.ERR_ARG, c2.ERR_ARG, c2.ERR_DTYPE, c2.ERR_NULL, c2.ERR_NULL, c2.ERR_ARG]


def test_workspace_sizes():
    assert c2.conv2d_rms_norm_bwd_workspace_bytes(0, 8) == 0
    assert c2.conv2d_rms_norm_bwd_workspace_bytes(8, 16385) == 0
    for M in (1, 7, 1000, 1 << 20, TOP):
        for C in (1, 64, 1001, 16384):
            n = c2.conv2d_rms_norm_bwd_workspace_bytes(M, C)
            assert n >= 4 * C and n % 16 == 0
    for dtype in (c2.F32, c2.BF16):
        assert c2.conv2d_matmul_workspace_bytes(0, 1, 1, dtype) == 0
        assert c2.conv2d_matmul_workspace_bytes(8192, 8192, 8192, dtype) == 0   # enough tiles without splitting
        assert c2.conv2d_matmul_workspace_bytes(100, 8192, 64, dtype) > 0
        assert c2.conv2d_matmul_bwd_workspace_bytes(8192, 4096, 4096, dtype) >= 8192 * 4096 * 2
    assert c2.conv2d_matmul_workspace_bytes(100, 8192, 64, 7) == 0
    assert c2.conv2d_matmul_bwd_workspace_bytes(TOP, 1, 1, c2.BF16) == 0


# ------------------------------------------------------------------ the definitions

def test_words_of_the_generator():
    """The published answers of Philox4x32-10."""
    F = 0xFFFFFFFF
    for counter, key, want in [
            ([0, 0, 0, 0], [0, 0], [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
            ([F, F, F, F], [F, F], [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
            ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
             [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1])]:
        assert [int(v) for v in ref.philox(counter, key)] == want


def test_definition_of_dropout():
    keep = ref.dropout_keep(300, 1001, 0.3, 5, 6)
    assert abs(keep.mean() - 0.7) < 5 * np.sqrt(0.21 / keep.size)
    assert ref.dropout_keep(7, 5, 0.0, 1, 2).all()
    np.testing.assert_array_equal(ref.dropout_keep(2, 9, 0.5, 1, 2, row0=5), ref.dropout_keep(7, 1001, 0.5, 1, 2)[5:, :9])


@pytest.mark.parametrize("act", [0, 2, 3])
def test_definition_gradients_match_differences(act):
    rng = np.random.default_rng(act)
    h = 1e-6
    x, w, b = rng.standard_normal((5, 7)), rng.standard_normal((4, 7)), rng.standard_normal(4)
    dy = rng.standard_normal((5, 4))
    z = ref.matmul(x, w, b, None, act)[1]
    grads = dict(zip("xwb", ref.matmul_bwd(dy, z, x, w, act)))
    f = lambda **k: (ref.matmul(k.get("x", x), k.get("w", w), k.get("b", b), None, act)[0] * dy).sum()  # noqa: E731
    for name, at in dict(x=x, w=w, b=b).items():
        v = rng.standard_normal(at.shape)
        want = (f(**{name: at + h * v}) - f(**{name: at - h * v})) / (2 * h)
        assert abs((grads[name] * v).sum() - want) < 1e-6
    g, dh = 1 + 0.2 * rng.standard_normal(7), rng.standard_normal((5, 7))
    dy = rng.standard_normal((5, 7))
    _, _, rstd = ref.rms_norm(x, None, g, 1e-5)
    dx, dg = ref.rms_norm_bwd(dy, dh, x, g, rstd)
    f = lambda x, g: (ref.rms_norm(x, None, g, 1e-5)[1] * dy).sum() + (x * dh).sum()  # noqa: E731
    v, u = rng.standard_normal(x.shape), rng.standard_normal(7)
    assert abs((dx * v).sum() - (f(x + h * v, g) - f(x - h * v, g)) / (2 * h)) < 1e-6
    assert abs((dg * u).sum() - (f(x, g + h * u) - f(x, g - h * u)) / (2 * h)) < 1e-6
