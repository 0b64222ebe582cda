"""Gradients of gamma and beta over many images: the images' sums, all of one
sign and size, are added in fp64 in every form of the backward pass.
"""
import sys

import numpy as np
import pytest

import test_group_norm_gpu as small
from helpers import ensure_built, gpu_available
from oracle import operators as ref

pytestmark = pytest.mark.gpu

if gpu_available():
    ensure_built()
    import torch
    import cnn_convolution_conv2d_amd as c2

U = small.U


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


#                 N      C    H  W  G   dtype
@pytest.mark.parametrize("N,C,H,W,G,dtype", [(30000, 32, 1, 2, 4, "f32"),    # a group in registers
                                             (40000, 18, 2, 1, 9, "f32"),    # two launches
                                             (50000, 32, 3, 3, 4, "f32")])   # chunks that exchange their sums
def test_many_images(N, C, H, W, G, dtype):
    """dy is 0.1 throughout: a run of fp32 additions would drift to one side, by
    thousands of u.  An image's own sum of at most 9 values is off by 9 u, its
    normalised values by 8 u, the total by one rounding."""
    print("[many images]", N, C, H, W, G, dtype, file=sys.stderr, flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(C)
    P = H * W
    x = torch.randn(N, P, C, generator=gen, device="cuda") + 2 * torch.arange(C, device="cuda")
    dy = torch.full_like(x, 0.1)
    mean, rstd = torch.empty(N, G, device="cuda"), torch.empty(N, G, device="cuda")
    dx, dg, db = torch.empty_like(x), torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    n = c2.conv2d_group_norm_workspace_bytes(N, C, H, W, G, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    c2.conv2d_group_norm_nhwc(x, None, None, dx, mean, rstd, ws, n, N, C, H, W, G, C, C, small.EPS, c2.F32, 0)
    c2.conv2d_group_norm_bwd_nhwc(dy, x, None, None, mean, rstd, dx, dg, db, ws, n, N, C, H, W, G, C, C, C, c2.F32, 0)
    mu, r = mean.cpu().numpy().astype(np.float64), rstd.cpu().numpy().astype(np.float64)
    xh = ref.normalise(x.cpu().numpy(), mu, r)
    step = float(np.float32(0.1))
    want, size = step * xh.sum(axis=(0, 1)), step * np.abs(xh).sum(axis=(0, 1))
    small.inside(db.cpu().numpy(), np.full(C, step * N * P), 10 * U * step * N * P, "dbeta")
    small.inside(dg.cpu().numpy(), want, 18 * U * size, "dgamma")
