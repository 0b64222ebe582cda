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
