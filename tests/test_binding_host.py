"""The C extension that passes the operators' arguments (no GPU: every call here
is refused before anything is enqueued)."""
import numpy as np
import pytest
import torch

from helpers import ensure_built

ensure_built()
import cnn_convolution_conv2d_amd as c2  # noqa: E402


def rows(x, q, scale, M=1, K=1, ldx=1, ldq=1, dtype=c2.BF16):
    c2.conv2d_quantize_rows(x, q, scale, M, K, ldx, ldq, dtype, stream=0)


def test_the_first_bad_argument_is_the_one_blamed():
    t = torch.zeros(4)
    with pytest.raises(AttributeError, match="ndarray"):
        rows(np.zeros(4, np.float32), t, t)
    with pytest.raises(AttributeError, match="'list'"):
        rows(t, [1], t, M=1 << 40)
    with pytest.raises(OverflowError, match="C int"):
        rows(t, t, t, M=1 << 40, K=2.5)
    with pytest.raises(TypeError):
        rows(t, t, t, M=2.5, K=1 << 40)


def test_a_count_that_does_not_match_is_refused():
    with pytest.raises(TypeError, match="quantize_rows takes 10 arguments, got 2"):
        c2._binding.quantize_rows(c2._quantize_rows, None)


def test_addresses_and_tensors_are_the_same():
    t = torch.zeros(4)
    for x in (t, t.data_ptr()):
        with pytest.raises(c2.Conv2dError) as e:
            rows(x, t, None)
        assert e.value.code == c2.ERR_NULL


@pytest.fixture
def without_extension(tmp_path, monkeypatch):
    """The package as it loads where no extension is built for this Python."""
    import importlib.util
    import os
    import shutil
    src = os.path.dirname(c2.__file__)
    shutil.copy(os.path.join(src, "__init__.py"), tmp_path)
    open(tmp_path / "_binding.so", "w").close()   # another Python's
    monkeypatch.setenv("CONV2D_LIBRARY", c2.LIB_PATH)
    spec = importlib.util.spec_from_file_location("without_extension", tmp_path / "__init__.py")
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_the_package_works_without_the_extension(without_extension):
    w = without_extension
    assert w.conv2d_out_dim(9, 3, 1, 1, 1) == 9
    t = torch.zeros(64)
    size = (2, 32, 5, 7, 4)
    for mod in (c2, w):
        codes = []
        for call in (lambda: mod.conv2d_quantize_rows(t, t, None, 1, 1, 1, 1, c2.BF16, stream=0),
                     lambda: mod.conv2d_quantize_rows(t, t, t, 1, 0, 1, 1, c2.BF16, stream=0),
                     lambda: mod.conv2d_int8_matmul(t, t, t, t, None, t, None, 0, 1, 1, 1, 1, 1, 1, 7, 0, stream=0),
                     lambda: mod.conv2d_group_norm_nhwc(t, t, None, t, t, t, t, 8, *size, 32, 32, 1e-5, 1, 0, stream=0),
                     lambda: mod.conv2d_group_norm_nhwc(t, t, None, t, t, t, t, 8, *size, 32, 32, -1.0, 1, 0, stream=0),
                     lambda: mod.conv2d_group_norm_quant_nhwc(t, t, t, t, None, t, t, t, 8, *size, 32, 32, 1e-5, 1, 0,
                                                              stream=0),
                     lambda: mod.conv2d_group_norm_bwd_nhwc(t, t, t, t, t, None, t, t, t, t, 8, *size, 32, 32, 32, 1, 0,
                                                            stream=0)):
            with pytest.raises(mod.Conv2dError) as e:
                call()
            codes.append(e.value.code)
        assert codes == [c2.ERR_NULL, c2.ERR_ARG, c2.ERR_DTYPE, c2.ERR_ARG, c2.ERR_ARG, c2.ERR_NULL, c2.ERR_NULL]
    with pytest.raises(TypeError, match="quantize_rows takes 10 arguments, got 2"):
        w._binding.quantize_rows(0, None)


def test_the_extension_is_named_for_its_python():
    import sysconfig
    from helpers import builder
    b = builder()
    assert b.BINDING.endswith("_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
    assert c2._binding.__file__ == b.BINDING


def test_a_build_without_python_headers(tmp_path, monkeypatch, capsys):
    """hipcc alone is enough; a library without the extension is then not stale."""
    from helpers import builder
    b = builder()
    monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    b._build_binding()
    assert not (tmp_path / "_binding.so").exists() and "ctypes" in capsys.readouterr().err
    assert not b.stale()
    monkeypatch.setattr(b, "has_python_headers", lambda: True)
    assert b.stale()


def test_hipcc_compiles_the_extension_where_there_is_no_gcc(tmp_path, monkeypatch):
    from helpers import builder
    b = builder()
    if not b.has_python_headers():
        pytest.skip("no Python.h")
    monkeypatch.setattr(b.shutil, "which", lambda name: None)
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    b._build_binding()
    import importlib.util
    spec = importlib.util.spec_from_file_location("_binding", tmp_path / "_binding.so")
    spec.loader.exec_module(importlib.util.module_from_spec(spec))
