"""Group norm on tensors large enough that workgroups exchange partial sums,
against the plain fp64 definitions, with the tolerances of the small ones: a
chunk's run of values is at most 16 long, then come trees and one value a
chunk, fewer than 64 roundings on any value's way.

Every case runs twice: as a caller has it, and with a wait limit of 0, which
makes workgroups compute the partial sums that they miss themselves.  The two
have to agree bit for bit.
"""
import sys

import numpy as np
import pytest

import test_group_norm_gpu as small
from helpers import ensure_built, gpu_available

pytestmark = pytest.mark.gpu

if gpu_available():
    ensure_built()
    import torch
    import cnn_convolution_conv2d_amd as c2


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")
    limit = c2.conv2d_set_wait_limit(64)
    yield
    c2.conv2d_set_wait_limit(limit)


def say(what):
    print(f"[large group norm] {what}", file=sys.stderr, flush=True)


def both_ways(run, outputs):
    """run() at the usual limit and at 0; the outputs of the first."""
    run()
    torch.cuda.synchronize()
    first = [t.clone() for t in outputs]
    for t in outputs:
        t.fill_(0)
    limit = c2.conv2d_set_wait_limit(0)
    run()
    torch.cuda.synchronize()
    c2.conv2d_set_wait_limit(limit)
    for a, b in zip(first, outputs):
        assert torch.equal(a, b), "the wait limit changes bits"


#           N    C    H    W    G  dtype   pad
FORWARD = [(3, 144, 131, 113, 9, "bf16", 0),    # 18 vectors a pixel, idle threads, a last chunk that is not full
           (200, 16, 45, 45, 2, "bf16", 8),     # one chunk an image, wider rows
           (1, 512, 113, 115, 4, "bf16", 0),    # the widest pixel, one image
           (2, 36, 211, 209, 3, "f32", 4)]


@pytest.mark.parametrize("N,C,H,W,G,dtype,pad", FORWARD)
def test_forward(N, C, H, W, G, dtype, pad):
    for act in (2, 1):
        say((N, C, H, W, G, dtype, pad, act))
        c = small.Case(N, C, H, W, G, act, dtype, pad=pad)
        both_ways(c.forward, [c.y.view, c.mean, c.rstd])
        if act == 2:
            small.check_forward(c, "forward")
    # in place, and a value that is not finite stays in its group
    want, x = c.y.view.clone(), c.x.view.clone()
    cg, P = C // G, H * W
    for limit in (64, 0):
        c2.conv2d_set_wait_limit(limit)
        c.x.view.copy_(x)
        c.x.view[P // 2, cg * (G - 1)] = float("inf")
        ws, n = c.workspace()
        c2.conv2d_group_norm_nhwc(c.x.view, c.gd, c.bd, c.x.view, None, None, ws, n, N, C, H, W, G, c.ld, c.ld,
                                  small.EPS, small.lt(dtype), 1)
        bad = c.x.view[:P, cg * (G - 1):]
        assert bool(bad.isnan().all())
        bad.copy_(want[:P, cg * (G - 1):])
        assert torch.equal(c.x.view, want)


@pytest.mark.parametrize("N,C,H,W,G,dtype", [(3, 144, 173, 171, 9, "bf16"), (40, 64, 51, 50, 32, "f32")])
def test_quantised(N, C, H, W, G, dtype):
    say((N, C, H, W, G, dtype))
    c = small.Case(N, C, H, W, G, 2, dtype)
    q = small.Padded(N * H * W, C, C, 0, torch.int8, 77)
    s = torch.full((N * H * W,), float("nan"), device="cuda")

    def run():
        ws, n = c.workspace()
        c2.conv2d_group_norm_quant_nhwc(c.x.view, c.gd, c.bd, q.view, s, c.mean, c.rstd, ws, n, N, C, H, W, G, c.ld, C,
                                        small.EPS, small.lt(dtype), 2)

    both_ways(run, [q.view, s, c.mean, c.rstd])
    small.check_quantised(c, q, s, "quantised")


@pytest.mark.parametrize("N,C,H,W,G,dtype", [(5, 136, 193, 193, 17, "bf16"), (3, 36, 341, 343, 9, "f32")])
def test_backward(N, C, H, W, G, dtype):
    say((N, C, H, W, G, dtype))
    c = small.Case(N, C, H, W, G, 2, dtype)
    c.forward()
    dg, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")

    def run(dx=None):
        ws, n = c.workspace(True)
        c2.conv2d_group_norm_bwd_nhwc(c.dy.view, c.x.view, c.gd, c.bd, c.mean, c.rstd, c.y.view if dx is None else dx,
                                      dg, db, ws, n, N, C, H, W, G, c.ld, c.ld, c.ld, small.lt(dtype), 2)

    both_ways(run, [c.y.view, dg, db])
    small.check_backward(c, dg, db, "backward")
    dy = c.dy.view.clone()
    for limit in (64, 0):   # dx over dy
        c2.conv2d_set_wait_limit(limit)
        c.dy.view.copy_(dy)
        run(c.dy.view)
        assert torch.equal(c.dy.view, c.y.view)


def test_replays_of_a_graph():
    """The workspace holds anything before every replay."""
    N, C, H, W, G = 3, 144, 173, 171, 9
    c = small.Case(N, C, H, W, G, 1, "bf16")
    ws, n = c.workspace(True)
    q = torch.empty(N * H * W, C, dtype=torch.int8, device="cuda")
    s = torch.empty(N * H * W, device="cuda")

    def step():
        c2.conv2d_group_norm_nhwc(c.x.view, c.gd, c.bd, c.y.view, c.mean, c.rstd, ws, n, N, C, H, W, G, C, C, small.EPS,
                                  c2.BF16, 1)
        c2.conv2d_group_norm_quant_nhwc(c.x.view, c.gd, c.bd, q, s, None, None, ws, n, N, C, H, W, G, C, C, small.EPS,
                                        c2.BF16, 1)

    step()
    torch.cuda.synchronize()
    out = (c.y.view, c.mean, c.rstd, q, s)
    want = [t.clone() for t in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        for t in out:
            t.fill_(0)
        ws.fill_(85 * k)
        c.x.view.add_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls that share the device wait for, and help, their own workgroups only."""
    cases = [small.Case(6, 128, 97, 99, 16, 1, "bf16", seed=k) for k in range(3)]
    want = []
    for c in cases:
        c.forward()
        want.append(c.host(c.y))
        c.y.view.fill_(0)
    spaces = [c.workspace() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        for c, (ws, n), st in zip(cases, spaces, streams):
            c2.conv2d_group_norm_nhwc(c.x.view, c.gd, c.bd, c.y.view, c.mean, c.rstd, ws, n, c.N, c.C, c.H, c.W, c.G,
                                      c.ld, c.ld, small.EPS, c2.BF16, 1, st)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        np.testing.assert_array_equal(c.host(c.y), w)


# rows that 16-byte vectors do not divide or are not aligned to, read in such
# vectors all the same where the tensor is large
#          N   C   H    W   G  dtype  pad skip
RAGGED = [(9, 531, 31, 29, 9, "bf16", 0, 0), (40, 9, 109, 107, 1, "bf16", 2, 1), (5, 258, 41, 40, 2, "f32", 1, 3),
          (3, 2051, 27, 26, 7, "bf16", 0, 0)]


@pytest.mark.parametrize("N,C,H,W,G,dtype,pad,skip", RAGGED)
def test_ragged_rows(N, C, H, W, G, dtype, pad, skip):
    say((N, C, H, W, G, dtype, pad, skip))
    c = small.Case(N, C, H, W, G, 2, dtype, pad=pad, skip=skip)
    c.forward()
    small.check_forward(c, "forward")
    dg, db = small.backward(c)
    small.check_backward(c, dg, db, "backward")
    assert c.y.untouched()
    ws, n = c.workspace()
    q = small.Padded(N * H * W, C, C + 1, 3, torch.int8, 77)
    s = torch.full((N * H * W,), float("nan"), device="cuda")
    c2.conv2d_group_norm_quant_nhwc(c.x.view, c.gd, c.bd, q.view, s, c.mean, c.rstd, ws, n, N, C, H, W, G, c.ld, C + 1,
                                    small.EPS, small.lt(dtype), 2)
    small.check_quantised(c, q, s, "quantised")
    # x over itself, which takes other vectors: the same fp64 values
    e = c.errors()
    c2.conv2d_group_norm_nhwc(c.x.view, c.gd, c.bd, c.x.view, None, None, ws, n, N, C, H, W, G, c.ld, c.ld, small.EPS,
                              small.lt(dtype), 2)
    small.inside(c.host(c.x), e["y"], e["e_y"] + small.HALF[dtype] * (np.abs(e["y"]) + e["e_y"]), "in place")
    assert c.x.untouched()
