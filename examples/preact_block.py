"""A pre-activation bottleneck block on channels-last bf16 activations, as it
is served with 8-bit weights, and the tuning of a norm's parameters.

    python examples/preact_block.py              serve: one block in a graph, checked against fp64, timed
    python examples/preact_block.py --train 20   tune gamma and beta of a norm by 20 gradient steps

The block:

    h = conv1x1_int8(silu(group_norm(x)))        C -> C/4
    h = conv3x3_bf16(silu(group_norm(h)))        C/4 -> C/4
    y = x + conv1x1_int8(silu(group_norm(h)))    C/4 -> C

A 1x1 convolution over channels-last pixels is a product of rows, so the
quantised group norm writes what the integer product reads.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import cnn_convolution_conv2d_amd as c2  # noqa: E402

EPS = 1e-5


class Int8Weight:
    """[out][in] fp32 weights as int8 rows with a scale for each."""

    def __init__(self, w):
        self.out, self.cin = w.shape
        self.q = torch.empty(self.out, self.cin, dtype=torch.int8, device="cuda")
        self.scale = torch.empty(self.out, device="cuda")
        c2.conv2d_quantize_rows(w, self.q, self.scale, self.out, self.cin, self.cin, self.cin, c2.F32)


class Norm:
    def __init__(self, gen, C, G):
        self.C, self.G = C, G
        self.gamma = 1 + 0.1 * torch.randn(C, generator=gen, device="cuda")
        self.beta = 0.1 * torch.randn(C, generator=gen, device="cuda")


class Block:
    def __init__(self, N, H, W, C, G, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.N, self.H, self.W, self.C, self.mid, self.M = N, H, W, C, C // 4, N * H * W
        self.norms = [Norm(gen, C, G), Norm(gen, self.mid, G), Norm(gen, self.mid, G)]
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        self.w1 = Int8Weight(rand(self.mid, C) / C ** 0.5)
        self.w3 = Int8Weight(rand(C, self.mid) / self.mid ** 0.5)
        self.w2 = (rand(self.mid, self.mid, 3, 3) / (9 * self.mid) ** 0.5).bfloat16()
        self.w2_packed = torch.empty(c2.conv2d_packed_weight_bytes(self.mid, self.mid, 3, 3, 1, c2.BF16),
                                     dtype=torch.uint8, device="cuda")
        c2.conv2d_pack_weights(self.w2, self.w2_packed, self.mid, self.mid, 3, 3, 1, c2.BF16)
        # buffers that every call uses
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.q = torch.empty(self.M, C, dtype=torch.int8, device="cuda")
        self.q_scale = torch.empty(self.M, device="cuda")
        self.h1, self.h2, self.h3 = (torch.empty(N, H, W, self.mid, **bf) for _ in range(3))
        self.y = torch.empty(N, H, W, C, **bf)
        sizes = [c2.conv2d_group_norm_workspace_bytes(N, n.C, H, W, n.G) for n in self.norms]
        sizes += [c2.conv2d_int8_matmul_workspace_bytes(self.M, w.cin, w.out) for w in (self.w1, self.w3)]
        self.workspace = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")

    def norm(self, n, x, y):
        c2.conv2d_group_norm_nhwc(x, n.gamma, n.beta, y, None, None, self.workspace, self.workspace.numel(), self.N,
                                  n.C, self.H, self.W, n.G, n.C, n.C, EPS, c2.BF16, c2.ACT_SILU)

    def norm_1x1(self, n, x, w, y):
        ws, size = self.workspace, self.workspace.numel()
        c2.conv2d_group_norm_quant_nhwc(x, n.gamma, n.beta, self.q, self.q_scale, None, None, ws, size, self.N, n.C,
                                        self.H, self.W, n.G, n.C, n.C, EPS, c2.BF16, c2.ACT_SILU)
        c2.conv2d_int8_matmul(self.q, self.q_scale, w.q, w.scale, None, y, ws, size, self.M, w.cin, w.out, w.cin,
                              w.cin, w.out, c2.BF16, c2.EPI_NONE)

    def __call__(self, x):
        self.norm_1x1(self.norms[0], x, self.w1, self.h1)
        self.norm(self.norms[1], self.h1, self.h2)
        c2.conv2d_fwd_nhwc_packed(self.h2, self.w2_packed, None, self.h3, self.N, self.mid, self.H, self.W, self.mid,
                                  3, 3, 1, 1, 1, 1, c2.BF16, c2.EPI_NONE)
        self.norm_1x1(self.norms[2], self.h3, self.w3, self.y)
        return self.y.add_(x)

    def plain(self, x):
        """The block in fp64 on the host, without the 8-bit step of the activations."""
        def norm(n, v):
            u = v.reshape(v.shape[0], -1, n.G, n.C // n.G)
            mean = u.mean((1, 3), keepdim=True)
            var = (u - mean).square().mean((1, 3), keepdim=True)
            z = ((u - mean) / (var + EPS).sqrt()).reshape(v.shape) * n.gamma.cpu().double() + n.beta.cpu().double()
            return z * torch.sigmoid(z)

        w1, w3 = ((w.q.cpu().double() * w.scale.cpu().double()[:, None]).T for w in (self.w1, self.w3))
        x = x.cpu().double()
        h = norm(self.norms[1], norm(self.norms[0], x) @ w1)
        h = torch.nn.functional.conv2d(h.permute(0, 3, 1, 2), self.w2.cpu().double(), padding=1).permute(0, 2, 3, 1)
        return x + norm(self.norms[2], h) @ w3


def serve(N=2, H=28, W=28, C=256, G=16):
    """One block captured into a graph; returns its relative error (rms) against fp64."""
    block = Block(N, H, W, C, G)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.empty(N, H, W, C, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=gen)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(x)
    worst = 0.0
    for _ in range(3):   # new inputs through the same graph
        x.normal_(generator=gen)
        graph.replay()
        torch.cuda.synchronize()
        want = block.plain(x)
        worst = max(worst, float((block.y.cpu().double() - want).norm() / want.norm()))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"block of {N}x{H}x{W}x{C}: {begin.elapsed_time(end) * 10:.1f} us a replay, relative error {worst:.2e}")
    return worst


def train(steps, N=4, H=14, W=14, C=64, G=8, rate=0.5):
    """Fits gamma and beta so that silu(group_norm(x)) comes near another norm's output; returns the losses."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    x = torch.empty(N, H, W, C, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=gen)
    teacher, student = Norm(gen, C, G), Norm(gen, C, G)
    mean, rstd = (torch.empty(N, G, device="cuda") for _ in range(2))
    size = c2.conv2d_group_norm_workspace_bytes(N, C, H, W, G, backward=True)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    target, y, dx = (torch.empty_like(x) for _ in range(3))
    dgamma, dbeta = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")

    def forward(n, out):
        c2.conv2d_group_norm_nhwc(x, n.gamma, n.beta, out, mean, rstd, ws, size, N, C, H, W, G, C, C, EPS, c2.BF16,
                                  c2.ACT_SILU)

    forward(teacher, target)
    losses = []
    for _ in range(steps):
        forward(student, y)
        diff = y.float() - target.float()
        losses.append(0.5 * float(diff.square().sum()) / (N * H * W))
        dy = (diff / (N * H * W)).bfloat16()
        c2.conv2d_group_norm_bwd_nhwc(dy, x, student.gamma, student.beta, mean, rstd, dx, dgamma, dbeta, ws, size, N,
                                      C, H, W, G, C, C, C, c2.BF16, c2.ACT_SILU)
        student.gamma -= rate * dgamma
        student.beta -= rate * dbeta
    print(f"{steps} steps: loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    return losses


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--train", type=int, default=0, metavar="STEPS", help="tune a norm's parameters instead of serving")
    a = p.parse_args()
    train(a.train) if a.train else serve()


if __name__ == "__main__":
    main()
