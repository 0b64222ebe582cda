"""dgamma of the RMS norm and dbias of the products: the sums of a workgroup's groups of rows are added in fp64, so one
large value leaves the others their digits.  Every lane has one row here: a workgroup's sum is rounded to fp32 once, and
the output once."""
import numpy as np
import pytest

from helpers import ensure_built, gpu_available

pytestmark = pytest.mark.gpu

if gpu_available():
    ensure_built()
    import torch
    import cnn_convolution_conv2d_amd as c2
    from row_helpers import U, inside

# rows that one workgroup's lanes hold one of each, for the type's vectors
SIZES = [("f32", 256, 1), ("bf16", 256, 1), ("bf16", 256, 8), ("f32", 64, 16), ("bf16", 128, 16), ("f32", 4, 250)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


def values(dtype, M, C):
    """The first row 2^24, the others 1: in fp32, added one after the other, these would all be lost."""
    t, dt = (torch.float32, c2.F32) if dtype == "f32" else (torch.bfloat16, c2.BF16)
    dy = torch.ones(M, C, dtype=t, device="cuda")
    dy[0] = 2.0 ** 24
    return dy, np.full(C, 2.0 ** 24 + M - 1), t, dt


@pytest.mark.parametrize("dtype,M,C", SIZES)
def test_dgamma(dtype, M, C):
    dy, want, t, dt = values(dtype, M, C)
    h, dx = torch.ones(M, C, dtype=t, device="cuda"), torch.empty(M, C, dtype=t, device="cuda")
    rstd, dgamma = torch.ones(M, device="cuda"), torch.empty(C, device="cuda")
    n = c2.conv2d_rms_norm_bwd_workspace_bytes(M, C)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    c2.conv2d_rms_norm_bwd(dy, None, h, None, rstd, dx, dgamma, ws, n, M, C, C, 0, C, C, dt)
    inside(dgamma.cpu().numpy(), want, 2 * U * want, f"dgamma {dtype} {M}x{C}")


@pytest.mark.parametrize("dtype,M,C", SIZES)
def test_dbias(dtype, M, C):
    dy, want, t, dt = values(dtype, M, C)
    x, w = torch.ones(M, 8, dtype=t, device="cuda"), torch.ones(C, 8, dtype=t, device="cuda")
    db = torch.empty(C, device="cuda")
    n = c2.conv2d_matmul_bwd_workspace_bytes(M, 8, C, dt)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    c2.conv2d_matmul_bwd(dy, None, x, w, None, None, db, ws, n, M, 8, C, C, 0, 8, 8, 0, 0, dt, c2.ACT_NONE)
    inside(db.cpu().numpy(), want, 2 * U * want, f"dbias {dtype} {M}x{C}")
