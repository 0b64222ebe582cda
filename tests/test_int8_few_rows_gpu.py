"""Integer products of up to 64 rows with many channels or long rows: every
instance of the kernel that streams the weights (one or two groups of channels
a workgroup, 2, 4 or 8 steps in flight), with edges inside a group, a step and
a block of rows."""
import pytest

import test_int8_gpu as small
from helpers import gpu_available

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [17, 32, 33, 64])
@pytest.mark.parametrize("K,N", [(16, 8192), (208, 8201), (1296, 8223)])
def test_many_channels(M, K, N, dtype):
    small.run_product(M, K, N, dtype, bias=M % 2 == 0, relu=N % 2 == 0)


@pytest.mark.parametrize("M", [1, 2, 16])
@pytest.mark.parametrize("K,N", [(2048, 16384), (4096, 16399), (2064, 4096), (6160, 2050), (16384, 48), (1024, 8192),
                                 (384, 16384)])
def test_long_rows(M, K, N):
    small.run_product(M, K, N, "bf16", relu=M == 2)


def test_strides_of_many_channels():
    small.run_product(40, 272, 8215, padq=16, padw=48, pady=5, skip=16)
    small.run_product(20, 272, 8215, "f32", padq=32, padw=16, pady=1, skip=32)
