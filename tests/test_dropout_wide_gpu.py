"""Dropout of rows as wide as an int counts: the mask equals the definition's at the row's start, middle and end."""
import numpy as np
import pytest

from helpers import ensure_built, gpu_available
from oracle import operators as ref

pytestmark = pytest.mark.gpu

if gpu_available():
    ensure_built()
    import torch
    import cnn_convolution_conv2d_amd as c2


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


def keep(row, first, count, p, seed, offset):
    """Columns first .. of a row, first a multiple of 4."""
    groups = first // 4 + np.arange(-(-count // 4))
    words = ref.philox([groups, np.full_like(groups, row), offset, 0], [seed, 0])
    words = np.stack([np.broadcast_to(w, groups.shape) for w in words], axis=1).reshape(-1)[:count]
    return words >= np.uint64(int(p * 2.0 ** 32))


# 2^31 - 1 and 2^31 - 7 columns: the count of vectors and the end of the last one pass 2^31
@pytest.mark.parametrize("dtype,M,C", [("bf16", 1, (1 << 31) - 1), ("f32", 1, (1 << 31) - 1), ("bf16", 2, (1 << 31) - 7),
                                       ("bf16", 1, (1 << 31) - 8)])
def test_widest_rows(dtype, M, C):
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    rng = torch.tensor([5, 9], device="cuda")
    x = torch.ones(M * C, dtype=t, device="cuda")
    y = torch.full((M * C + 64,), 7.0, dtype=t, device="cuda")
    c2.conv2d_dropout(x, None, y, rng, 0.5, M, C, C, 0, C, c2.F32 if dtype == "f32" else c2.BF16)
    assert (y[M * C:] == 7).all()
    for row in range(M):
        for first in (0, 1 << 30, (C - 4001) // 4 * 4):
            count = min(5000, C - first)
            got = y[row * C + first:row * C + first + count].float().cpu().numpy()
            np.testing.assert_array_equal(got, np.where(keep(row, first, count, 0.5, 5, 9), 2.0, 0.0))
    # nothing left as it was, in pieces that fit 32-bit counts
    for i in range(0, M * C, 1 << 30):
        assert not (y[i:min(i + (1 << 30), M * C)] == 7).any()
