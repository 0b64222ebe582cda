"""A residual block on rows (tokens, or channels-last pixels) in bf16, as it is
served and as it is trained.

    python examples/residual_block.py              serve: a batch and single rows in graphs, checked against fp64, timed
    python examples/residual_block.py --train 20   20 gradient steps in one graph, with a new dropout mask each

The block, on the sum h of its input and a residual:

    y = h + dropout(silu(rms_norm(h) w1^T + b1) w2^T + b2)      C -> F -> C

Serving needs no dropout, and the second product adds h in its epilogue.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import cnn_convolution_conv2d_amd as c2  # noqa: E402

EPS = 1e-5


class Block:
    """Parameters, gradients and the buffers of M rows."""

    def __init__(self, M, C, F, p=0.1, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.M, self.C, self.F, self.p = M, C, F, p
        self.gamma = 1 + 0.1 * rand(C)
        self.w1, self.b1 = (rand(F, C) / C ** 0.5).bfloat16(), 0.1 * rand(F)
        self.w2, self.b2 = (rand(C, F) / F ** 0.5).bfloat16(), 0.1 * rand(C)
        self.rng = torch.tensor([seed, 0], device="cuda")   # the mask's seed and offset
        self.grads = {n: torch.empty_like(getattr(self, n)) for n in ("gamma", "w1", "b1", "w2", "b2")}
        rows = lambda n: torch.empty(M, n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.h, self.n, self.o, self.y, self.dx = (rows(C) for _ in range(5))
        self.z, self.a, self.da = (rows(F) for _ in range(3))
        self.rstd = torch.empty(M, device="cuda")
        size = max(c2.conv2d_rms_norm_bwd_workspace_bytes(M, C),
                   *(f(M, k, n, c2.BF16) for k, n in ((C, F), (F, C))
                     for f in (c2.conv2d_matmul_workspace_bytes, c2.conv2d_matmul_bwd_workspace_bytes)))
        self.ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")

    def norm(self, x, residual):
        M, C = self.M, self.C
        c2.conv2d_rms_norm(x, residual, self.gamma, self.h, self.n, self.rstd, M, C, C, C, C, C, EPS, c2.BF16)

    def product(self, x, w, bias, residual, z, y, act):
        N, K = w.shape
        c2.conv2d_matmul(x, w, bias, residual, z, y, self.ws, self.ws.numel(), self.M, K, N, K, K, N, N, N, c2.BF16, act)

    def product_bwd(self, dy, z, x, w, dx, dw, db, act):
        N, K = w.shape
        c2.conv2d_matmul_bwd(dy, z, x, w, dx, dw, db, self.ws, self.ws.numel(), self.M, K, N, N, N, K, K, K, K, c2.BF16, act)

    def dropout(self, x, residual, y):
        c2.conv2d_dropout(x, residual, y, self.rng, self.p, self.M, self.C, self.C, self.C, self.C, c2.BF16)

    def serve(self, x, residual):
        self.norm(x, residual)
        self.product(self.n, self.w1, self.b1, None, None, self.a, c2.ACT_SILU)
        self.product(self.a, self.w2, self.b2, self.h, None, self.y, c2.ACT_NONE)
        return self.y

    def forward(self, x, residual):
        self.norm(x, residual)
        self.product(self.n, self.w1, self.b1, None, self.z, self.a, c2.ACT_SILU)
        self.product(self.a, self.w2, self.b2, None, None, self.o, c2.ACT_NONE)
        self.dropout(self.o, self.h, self.y)
        return self.y

    def backward(self, dy):
        """The gradient of x and of the residual alike; the parameters' are in self.grads."""
        g = self.grads
        self.dropout(dy, None, self.o)   # do, over what is not needed again
        self.product_bwd(self.o, None, self.a, self.w2, self.da, g["w2"], g["b2"], c2.ACT_NONE)
        self.product_bwd(self.da, self.z, self.n, self.w1, self.dx, g["w1"], g["b1"], c2.ACT_SILU)
        c2.conv2d_rms_norm_bwd(self.dx, dy, self.h, self.gamma, self.rstd, self.dx, g["gamma"], self.ws, self.ws.numel(),
                               self.M, self.C, self.C, self.C, self.C, self.C, c2.BF16)
        return self.dx

    def plain(self, x, residual, keep=None):
        """The block in fp64 on the host (autograd tracks the parameters): y, the leaves."""
        leaf = {n: getattr(self, n).cpu().double().requires_grad_() for n in self.grads}
        leaf["x"], r = x.cpu().double().requires_grad_(), residual.cpu().double()
        h = leaf["x"] + r
        n = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * leaf["gamma"]
        z = n @ leaf["w1"].T + leaf["b1"]
        o = (z * torch.sigmoid(z)) @ leaf["w2"].T + leaf["b2"]
        return h + (o if keep is None else torch.where(keep, o / (1 - self.p), torch.zeros_like(o))), leaf


def captured(fn):
    """fn as a graph, after a first call on a side stream."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn()
    return graph


def inputs(M, C, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return [torch.randn(M, C, generator=gen, device="cuda").bfloat16() for _ in range(3)]


def relative(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


def serve(M=1, C=1024, F=4096):
    """The block in a graph; returns its relative error (rms) against fp64."""
    block = Block(M, C, F)
    x, r, _ = inputs(M, C, 1)
    graph = captured(lambda: block.serve(x, r))
    worst = 0.0
    for seed in (2, 3):   # new inputs through the same graph
        for t, v in zip((x, r), inputs(M, C, seed)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        with torch.no_grad():
            worst = max(worst, relative(block.y, block.plain(x, r)[0]))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"block of {M} rows, {C} -> {F} -> {C}: {begin.elapsed_time(end) * 10:.1f} us a replay, relative error {worst:.2e}")
    return worst


def gradients(M=300, C=256, F=512, keep=None):
    """Relative errors of y and of every gradient of sum(y dy) against fp64 autograd.
    keep(M, C, p, seed, offset): the mask that the dropout's counter gives."""
    block = Block(M, C, F)
    x, r, dy = inputs(M, C, 5)
    block.rng[1] = 7
    block.forward(x, r)
    block.backward(dy)
    seed, offset = block.rng.tolist()
    y, leaf = block.plain(x, r, torch.from_numpy(keep(M, C, block.p, seed, offset)))
    y.backward(dy.cpu().double())
    errors = {n: relative(g, leaf[n].grad) for n, g in block.grads.items()}
    errors.update(x=relative(block.dx, leaf["x"].grad), y=relative(block.y, y.detach()))
    return errors


def train(steps, M=512, C=256, F=512, rate=0.005):
    """Fits the block to another one's outputs; a step is one replay.  Returns the losses."""
    teacher, block = Block(M, C, F, p=0.0, seed=1), Block(M, C, F, seed=2)
    x, r, dy = inputs(M, C, 6)
    target = teacher.forward(x, r).clone()

    def step():
        block.rng[1].add_(1)   # a new mask at every replay
        dy.copy_((block.forward(x, r).float() - target.float()) * (2 / M))
        block.backward(dy)
        for n, g in block.grads.items():
            getattr(block, n).sub_(g, alpha=rate)

    start = {n: getattr(block, n).clone() for n in block.grads}
    graph = captured(step)
    for n, v in start.items():
        getattr(block, n).copy_(v)
    losses = []
    for _ in range(steps):
        graph.replay()
        losses.append(float((block.y.float() - target.float()).square().sum(1).mean()))
    print(f"{steps} steps: loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    return losses


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--train", type=int, default=0, metavar="STEPS", help="train the block instead of serving it")
    a = p.parse_args()
    if a.train:
        train(a.train)
    else:
        for M in (1, 2048):
            serve(M)


if __name__ == "__main__":
    main()
