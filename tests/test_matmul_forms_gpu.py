"""Every kernel form of the products (tests/product_forms.py) against the plain fp64 definitions: whole numbers, whose
sums are exact, and normal values with an activation, by the helpers and tolerances of tests/test_matmul_gpu.py."""
import pytest

import product_forms as pf
from helpers import gpu_available

pytestmark = pytest.mark.gpu

if gpu_available():
    from test_matmul_gpu import run_backward, run_forward


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("kind,M,K,N,dtype,pad,name", pf.FORMS, ids=lambda v: str(v).replace(" ", "-"))
def test_form(kind, M, K, N, dtype, pad, name):
    if kind == "forward":
        run_forward(M, K, N, dtype, ints=True, act=1, z=True, padx=pad, padw=pad, pad=pad)
        run_forward(M, K, N, dtype, act=2, z=False, residual=False, padx=pad, padw=pad)
    else:
        run_backward(M, K, N, dtype, act=1, ints=True, want=(kind,), padx=pad, padw=pad, pad=pad)
        run_backward(M, K, N, dtype, act=3, want=(kind,), padx=pad, padw=pad)
