"""The example of a residual block that runs the row operators together."""
import importlib.util
import os

import numpy as np
import pytest

from helpers import ensure_built, gpu_available
from oracle import operators as ref

pytestmark = pytest.mark.gpu

if gpu_available():
    ensure_built()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "residual_block.py")
    spec = importlib.util.spec_from_file_location("residual_block", path)
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


# A value passes at most 8 roundings to bf16 on its way (h, n, z, a and the output; going back do, da, dz, dx), each of
# 2^-8 of it at most: with independent signs the root of their squares' sum stays below 8 / sqrt(3) 2^-8 = 1.8%
BOUND = 8 * 2.0 ** -8 / 3 ** 0.5


@pytest.mark.parametrize("M,C,F", [(1, 1024, 4096), (7, 200, 333), (300, 256, 512)])
def test_serving(M, C, F):
    assert block.serve(M, C, F) < BOUND


@pytest.mark.parametrize("M,C,F", [(300, 256, 512), (33, 72, 136), (65, 77, 131), (1, 64, 64)])
def test_gradients(M, C, F):
    errors = block.gradients(M, C, F, keep=ref.dropout_keep)
    assert set(errors) == {"gamma", "w1", "b1", "w2", "b2", "x", "y"}
    for name, error in errors.items():
        assert error < BOUND, (name, error)


def test_training_runs():
    losses = block.train(5)
    assert len(losses) == 5 and np.isfinite(losses).all()


def test_two_blocks_at_once():
    """Two blocks on two streams, each with its own workspace: the bits of each alone."""
    import torch
    blocks = [block.Block(600, 512, 1024, seed=s) for s in (1, 2)]
    data = [block.inputs(600, 512, s) for s in (3, 4)]
    want = []
    for b, (x, r, dy) in zip(blocks, data):
        b.forward(x, r)
        b.backward(dy)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (b.y, b.dx, *b.grads.values())])
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, (x, r, dy), s in zip(blocks, data, streams):
            with torch.cuda.stream(s):
                b.forward(x, r)
                b.backward(dy)
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        for got, t in zip((b.y, b.dx, *b.grads.values()), w):
            assert torch.equal(got, t)
