"""Row operators on streams, in graphs and in a training step, from buffers that hold nothing of an earlier call: every
output, intermediate and workspace is overwritten before each round, and two sets of inputs take turns, so that a value
read too early, left over or never written changes the result."""
import importlib.util
import os

import pytest

from helpers import ROOT, ensure_built, gpu_available

pytestmark = pytest.mark.gpu

if gpu_available():
    ensure_built()
    import torch
    import cnn_convolution_conv2d_amd as c2
    spec = importlib.util.spec_from_file_location("residual_block", os.path.join(ROOT, "examples", "residual_block.py"))
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


def spoil(tensors):
    for t in tensors:
        t.fill_(255 if t.dtype == torch.uint8 else float("nan"))


def same(got, want, what):
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), (what, i)


def buffers(b):
    return [b.h, b.n, b.o, b.y, b.dx, b.z, b.a, b.da, b.rstd, b.ws, *b.grads.values()]


def results(b):
    return [t.clone() for t in (b.y, b.dx, *b.grads.values())]


def both(b, data):
    x, r, dy = data
    b.forward(x, r)
    b.backward(dy)


def blocks(M=600, C=512, F=1024):
    """Two blocks, two sets of inputs for each, and the results of each set alone."""
    pair = [block.Block(M, C, F, seed=s) for s in (1, 2)]
    data = [[block.inputs(M, C, 10 * i + s) for s in (3, 4)] for i in range(2)]
    want = []
    for b, sets in zip(pair, data):
        want.append([])
        for d in sets:
            spoil(buffers(b))
            both(b, d)
            torch.cuda.synchronize()
            want[-1].append(results(b))
            assert all(bool(torch.isfinite(t).all()) for t in want[-1][-1])
    return pair, data, want


def test_two_blocks_on_two_streams():
    pair, data, want = blocks()
    streams = [torch.cuda.Stream() for _ in pair]
    for turn in range(6):
        for b in pair:
            spoil(buffers(b))
        torch.cuda.synchronize()
        for b, sets, s in zip(pair, data, streams):
            with torch.cuda.stream(s):
                both(b, sets[turn % 2])
        torch.cuda.synchronize()
        for b, w in zip(pair, want):
            same(results(b), w[turn % 2], turn)


def test_two_graphs_at_once():
    """A graph of each block, replayed on two streams together."""
    pair, data, want = blocks()
    fixed = [[t.clone() for t in sets[0]] for sets in data]
    graphs = [block.captured(lambda b=b, d=d: both(b, d)) for b, d in zip(pair, fixed)]
    streams = [torch.cuda.Stream() for _ in pair]
    for turn in range(6):
        for b, d, sets in zip(pair, fixed, data):
            spoil(buffers(b))
            for t, v in zip(d, sets[turn % 2]):
                t.copy_(v)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for b, w in zip(pair, want):
            same(results(b), w[turn % 2], turn)


def test_two_graphs_that_share_a_workspace():
    """One after the other on one stream, in either order."""
    pair, data, want = blocks()
    assert pair[0].ws.numel() == pair[1].ws.numel()
    pair[1].ws = pair[0].ws
    graphs = [block.captured(lambda b=b, d=d: both(b, d[0])) for b, d in zip(pair, data)]
    for order in ((0, 1), (1, 0), (0, 1)):
        for b in pair:
            spoil(buffers(b))
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for b, w in zip(pair, want):
            same(results(b), w[0], order)


# split along the sum; tiles of 256, of which dx and dw take those of 128; copied operands
@pytest.mark.parametrize("M,K,N,dtype", [(200, 2048, 136, "bf16"), (200, 2048, 136, "f32"), (4096, 1088, 4096, "bf16"),
                                         (2051, 1037, 2100, "bf16"), (24, 520, 8200, "bf16")])
def test_products_on_a_side_stream(M, K, N, dtype):
    t, dt = (torch.float32, c2.F32) if dtype == "f32" else (torch.bfloat16, c2.BF16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    put = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(t)  # noqa: E731
    w, b = put(N, K), put(N).float()
    sets = [(put(M, K), put(M, N)) for _ in range(2)]
    z, y, dx, dw, db = put(M, N), put(M, N), put(M, K), put(N, K), torch.empty(N, device="cuda")
    n = max(c2.conv2d_matmul_workspace_bytes(M, K, N, dt), c2.conv2d_matmul_bwd_workspace_bytes(M, K, N, dt), 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = (z, y, dx, dw, db)

    def step(x, dy, stream=None):
        c2.conv2d_matmul(x, w, b, dy, z, y, ws, n, M, K, N, K, K, N, N, N, dt, 2, stream)
        c2.conv2d_matmul_bwd(dy, z, x, w, dx, dw, db, ws, n, M, K, N, N, N, K, K, K, K, dt, 2, stream)

    want = []
    for x, dy in sets:
        spoil((*outs, ws))
        step(x, dy)
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
    side = torch.cuda.Stream()
    for turn in range(4):
        spoil((*outs, ws))
        torch.cuda.synchronize()
        step(*sets[turn % 2], side)
        side.synchronize()
        same(outs, want[turn % 2], turn)


@pytest.mark.parametrize("M,C,dtype", [(1, 4096, "bf16"), (300, 1001, "f32"), (3000, 256, "bf16"), (2000, 16384, "f32")])
def test_norm_and_dropout_on_a_side_stream(M, C, dtype):
    t, dt = (torch.float32, c2.F32) if dtype == "f32" else (torch.bfloat16, c2.BF16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    put = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(t)  # noqa: E731
    gamma, rng = 1 + 0.1 * torch.randn(C, generator=gen, device="cuda"), torch.tensor([3, 4], device="cuda")
    sets = [(put(M, C), put(M, C), put(M, C)) for _ in range(2)]
    h, y, dx, o = (put(M, C) for _ in range(4))
    q = torch.empty(M, C, dtype=torch.int8, device="cuda")
    q_scale, rstd, dgamma = (torch.empty(k, device="cuda") for k in (M, M, C))
    n = c2.conv2d_rms_norm_bwd_workspace_bytes(M, C)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = (h, y, rstd, q_scale, dx, dgamma, o)

    def step(x, r, dy, stream=None):
        c2.conv2d_rms_norm(x, r, gamma, h, y, rstd, M, C, C, C, C, C, 1e-5, dt, stream)
        c2.conv2d_rms_norm_quant(x, r, gamma, None, q, q_scale, None, M, C, C, C, 0, C, 1e-5, dt, stream)
        c2.conv2d_rms_norm_bwd(dy, r, h, gamma, rstd, dx, dgamma, ws, n, M, C, C, C, C, C, dt, stream)
        c2.conv2d_dropout(dx, y, o, rng, 0.3, M, C, C, C, C, dt, stream)

    want = []
    for s in sets:
        spoil((*outs, ws))
        q.fill_(-128)
        step(*s)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (*outs, q)])
    side = torch.cuda.Stream()
    for turn in range(4):
        spoil((*outs, ws))
        q.fill_(-128)
        torch.cuda.synchronize()
        step(*sets[turn % 2], side)
        side.synchronize()
        same((*outs, q), want[turn % 2], turn)


def test_training_in_a_graph_is_the_eager_steps(monkeypatch):
    """The example's training: its parameters and gradients after some replays are those of eager steps, bit by bit; every
    parameter has moved and the mask's offset went up once a step."""
    made = []

    class Kept(block.Block):
        def __init__(self, *a, **k):
            super().__init__(*a, **k)
            made.append(self)

    M, C, F, rate, steps = 200, 128, 256, 0.005, 4
    plain = block.Block
    monkeypatch.setattr(block, "Block", Kept)
    losses = block.train(steps, M, C, F, rate)
    teacher, trained = made
    eager = plain(M, C, F, seed=2)
    x, r, dy = block.inputs(M, C, 6)
    target = teacher.y   # its only pass's
    eager.rng[1] = 1     # the step before the capture, whose update is taken back
    for i in range(steps):
        before = {n: getattr(eager, n).clone() for n in eager.grads}
        eager.rng[1].add_(1)
        dy.copy_((eager.forward(x, r).float() - target.float()) * (2 / M))
        eager.backward(dy)
        for n, g in eager.grads.items():
            getattr(eager, n).sub_(g, alpha=rate)
            assert not torch.equal(getattr(eager, n), before[n]), (i, n)
        assert losses[i] == float((eager.y.float() - target.float()).square().sum(1).mean())
    assert trained.rng.tolist() == [2, 1 + steps]
    for n in eager.grads:
        assert torch.equal(getattr(trained, n), getattr(eager, n)), n
        assert torch.equal(trained.grads[n], eager.grads[n]), n
    same(results(trained), results(eager), "results")
