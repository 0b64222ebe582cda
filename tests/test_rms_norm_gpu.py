"""RMS norm with a residual (forward, in 8 bits, backward) on the GPU against the
plain fp64 definitions (oracle/operators.py).

With u = 2^-24: h is rounded to fp32 once (u) and to the output type.  A row's sum
of squares passes at most 16 fused additions in a lane, 6 steps over a wave and 15
over the waves: below 40 u of it with h's own rounding twice; rstd has half of
that, and a division, a root and a reciprocal: below 24 u.  y = h rstd gamma adds 3 u
and its rounding.  A backward sum has the same 37 additions of terms off by 3 u; dgamma
adds at most 512 rows in a lane and 256 lanes of a column.
"""
import sys

import numpy as np
import pytest

from helpers import ensure_built, gpu_available
from oracle import operators as ref

pytestmark = pytest.mark.gpu

if gpu_available():
    ensure_built()
    import torch
    import cnn_convolution_conv2d_amd as c2
    from row_helpers import HALF, TINY, U, Rows, inside, torch_type

EPS = 1e-5


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


def lt(dtype):
    return c2.F32 if dtype == "f32" else c2.BF16


class Case:
    def __init__(self, M, C, dtype, residual=True, gamma=True, pad=0, skip=0, seed=0, scale=1.0):
        rng = np.random.default_rng([seed, M, C])
        self.M, self.C, self.dtype = M, C, dtype
        put = lambda v, p: Rows(M, C, dtype, v, p, skip)  # noqa: E731
        spread = scale * np.exp(rng.standard_normal((M, 1)))
        self.x = put(spread * rng.standard_normal((M, C)), pad)
        self.r = put(spread * rng.standard_normal((M, C)), 2 * pad) if residual else None
        self.h, self.y, self.dx = put(None, 3 * pad), put(None, pad), put(None, 2 * pad)
        self.gamma = torch.from_numpy((1 + 0.3 * rng.standard_normal(C)).astype(np.float32)).cuda() if gamma else None
        self.rstd = torch.full((M,), 7.0, device="cuda")
        self.rng = rng
        self.what = f"M={M} C={C} {dtype} residual={residual} gamma={gamma} pad {pad} skip {skip}"
        print("[rms] " + self.what, file=sys.stderr, flush=True)

    def ld(self, *names):
        return [getattr(self, n).ld if getattr(self, n) is not None else 0 for n in names]

    def forward(self, stream=None):
        c2.conv2d_rms_norm(self.x, self.r, self.gamma, self.h, self.y, self.rstd, self.M, self.C,
                           *self.ld("x", "r", "h", "y"), EPS, lt(self.dtype), stream)

    def want(self):
        g = None if self.gamma is None else self.gamma.cpu().numpy()
        return ref.rms_norm(self.x.host(), None if self.r is None else self.r.host(), g, EPS)

    def check(self):
        h, y, rstd = self.want()
        half = HALF[self.dtype]
        inside(self.h.host(), h, (half + 2 * U) * np.abs(h) + TINY[self.dtype], self.what + " h")
        inside(self.rstd.cpu().numpy(), rstd, 24 * U * rstd, self.what + " rstd")
        inside(self.y.host(), y, (half + 30 * U) * np.abs(y) + TINY[self.dtype], self.what + " y")
        for t in (self.x, self.h, self.y):
            assert t.untouched(), self.what + ": wrote beside its rows"


SIZES = [(1, 1), (3, 2), (5, 3), (4, 7), (7, 8), (300, 9), (33, 16), (2, 64), (257, 100), (64, 256), (3, 511), (9, 513),
         (1, 1000), (4, 1001), (1, 4096), (2, 8192), (3, 8199), (2, 16384), (1500, 40), (1100, 1001), (1030, 4096),
         (1025, 2050), (1024, 12000), (1024, 16383)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,C", SIZES)
def test_forward(M, C, dtype):
    c = Case(M, C, dtype, residual=M % 3 != 0, gamma=C % 5 != 0)
    c.forward()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,skip", [(8, 8), (1, 0), (3, 1), (0, 3), (5, 5)])
def test_strides_and_alignment(pad, skip, dtype):
    for M, C in [(5, 64), (70, 333), (1027, 48), (3, 4097)]:
        c = Case(M, C, dtype, pad=pad, skip=skip)
        c.forward()
        c.check()
        check_backward(c)
        check_quantised(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_outputs_over_inputs_and_left_out(dtype):
    for M, C in [(3, 1000), (1100, 72), (2, 16384)]:
        for h, y in [("x", "r"), ("r", "x"), (None, "x"), ("r", None)]:
            c = Case(M, C, dtype)
            want = c.want()
            if h:
                c.h = getattr(c, h)
            if y:
                c.y = getattr(c, y)
            c.x_host = c.x.host()
            half = HALF[dtype]
            c.forward()
            inside(c.h.host(), want[0], (half + 2 * U) * np.abs(want[0]) + TINY[dtype], c.what + " h in place")
            inside(c.y.host(), want[1], (half + 30 * U) * np.abs(want[1]) + TINY[dtype], c.what + " y in place")
        c = Case(M, C, dtype)
        c.forward()
        y = c.y.host()
        c.y.store.fill_(7.0)
        c2.conv2d_rms_norm(c.x, c.r, c.gamma, None, c.y, None, M, C, *c.ld("x", "r"), 0, c.y.ld, EPS, lt(dtype))
        np.testing.assert_array_equal(c.y.host(), y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [5, 64, 1000, 5000])
def test_values_at_the_ends_of_the_range(C, dtype):
    """Squares beyond fp32's range on either side, a row of zeros, and rows that are not finite."""
    c = Case(8, C, dtype, residual=False)
    v = np.random.default_rng(C).standard_normal((8, C))
    v[0] *= 1e25
    v[1] = 3e38 * np.sign(v[1])
    v[2] *= 1e-25
    v[3] = 0
    v[4] *= 1e-12
    c.x.view.copy_(torch.from_numpy(v))
    c.forward()
    c.check()
    c2.conv2d_rms_norm(c.x, None, c.gamma, c.h, c.y, c.rstd, 8, C, *c.ld("x", "r", "h", "y"), 0.0, lt(dtype))
    _, y, rstd = ref.rms_norm(c.x.host()[[0, 1, 2, 4]], None, c.gamma.cpu().numpy(), 0.0)
    inside(c.y.host()[[0, 1, 2, 4]], y, (HALF[dtype] + 30 * U) * np.abs(y) + TINY[dtype], "eps 0")
    for bad in (np.nan, np.inf):
        c.x.view[5, C - 1] = bad
        c.x.view[7, 0] = bad
        c.forward()
        y = c.y.host()
        assert np.isnan(y[5, C - 1]) and np.isnan(y[7, 0])
        assert np.isfinite(y[[0, 1, 2, 3, 4, 6]]).all()
        assert (y[5, :C - 1] == 0).all() if bad == np.inf else np.isnan(y[5]).all()


# ------------------------------------------------------------------ in 8 bits


def quantise(c, h=True, stream=None):
    q, s = Rows(c.M, c.C, torch.int8, pad=c.y.ld - c.C, skip=3), torch.empty(c.M, device="cuda")
    c2.conv2d_rms_norm_quant(c.x, c.r, c.gamma, c.h if h else None, q, s, c.rstd, c.M, c.C, *c.ld("x", "r", "h"), q.ld,
                             EPS, lt(c.dtype), stream)
    return q, s


def check_quantised(c):
    q, s = quantise(c)
    h, y, rstd = c.want()
    t, scale = ref.quantise_rows(y)
    # y's own 30 u, the reciprocal and the product's rounding 3 u, of 127 at most
    inside(s.cpu().numpy(), scale, 33 * U * scale, c.what + " scale")
    inside(q.host(), t, 0.5 + 64 * U * 127, c.what + " q")
    inside(c.h.host(), h, (HALF[c.dtype] + 2 * U) * np.abs(h) + TINY[c.dtype], c.what + " h")
    inside(c.rstd.cpu().numpy(), rstd, 24 * U * rstd, c.what + " rstd")
    assert q.untouched() and c.h.untouched()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,C", SIZES)
def test_quantised(M, C, dtype):
    check_quantised(Case(M, C, dtype, residual=C % 3 != 0, gamma=M % 5 != 0))


def test_quantised_rows_that_are_not_finite():
    c = Case(5, 300, "bf16")
    c.x.view[1, 7], c.x.view[3, 299] = float("nan"), float("inf")
    q, s = quantise(c)
    assert np.isnan(s.cpu().numpy()).tolist() == [False, True, False, True, False]
    assert (q.host()[[1, 3]] == 0).all()


def test_quantised_then_product():
    """The 8-bit layer against fp64: half a step of every quantised value is the error that counts."""
    c = Case(150, 128, "bf16")
    N = 72
    rng = np.random.default_rng(3)
    wf = torch.from_numpy(rng.standard_normal((N, 128)).astype(np.float32)).cuda()
    w, ws = torch.empty(N, 128, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    c2.conv2d_quantize_rows(wf, w, ws, N, 128, 128, 128, c2.F32)
    q, s = quantise(c)
    y = torch.empty(150, N, device="cuda")
    n = c2.conv2d_int8_matmul_workspace_bytes(150, 128, N)
    wk = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    c2.conv2d_int8_matmul(q, s, w, ws, None, y, wk, n, 150, 128, N, q.ld, 128, N, c2.F32, 0)
    _, v, _ = c.want()
    wq = w.cpu().numpy().astype(np.float64) * ws.cpu().numpy().astype(np.float64)[:, None]
    _, scale = ref.quantise_rows(v)
    inside(y.cpu().numpy(), v @ wq.T, 0.505 * scale[:, None] * np.abs(wq).sum(axis=1), "norm + product")


# ------------------------------------------------------------------ backward


def check_backward(c, dh=True, dgamma=True, over=None):
    half = HALF[c.dtype]
    dy = Rows(c.M, c.C, c.dtype, c.rng.standard_normal((c.M, c.C)), c.x.ld - c.C, c.x.skip)
    d = Rows(c.M, c.C, c.dtype, c.rng.standard_normal((c.M, c.C)), c.h.ld - c.C, c.x.skip) if dh else None
    h = c.h.host()
    g = None if c.gamma is None else c.gamma.cpu().numpy()
    want, wg = ref.rms_norm_bwd(dy.host(), None if d is None else d.host(), h, g, c.rstd.cpu().numpy())
    dh_host = 0 if d is None else d.host()
    dx = dict(dy=dy, dh=d, h=c.h).get(over, c.dx)
    dg = torch.full((c.C,), 7.0, device="cuda") if dgamma else None
    n = c2.conv2d_rms_norm_bwd_workspace_bytes(c.M, c.C)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if dgamma else None
    t = dy.host() * (1 if g is None else g)
    xh = h * c.rstd.double().cpu().numpy()[:, None]
    yd = np.abs(dy.host() * xh)
    c2.conv2d_rms_norm_bwd(dy, d, c.h, c.gamma, c.rstd, dx, dg, ws, n if dgamma else 0, c.M, c.C, dy.ld,
                           d.ld if dh else 0, c.h.ld, dx.ld, lt(c.dtype))
    mean = np.abs(t * xh).mean(axis=1, keepdims=True)
    off = c.rstd.double().cpu().numpy()[:, None] * (4 * U * np.abs(t) + np.abs(xh) * 45 * U * mean) + 2 * U * (
        np.abs(want) + np.abs(dh_host))
    inside(dx.host(), want, off + half * (np.abs(want) + off) + TINY[c.dtype], c.what + " dx")
    assert dx.untouched()
    if dgamma:
        inside(dg.cpu().numpy(), wg, (min(c.M, 512) + 260) * U * yd.sum(axis=0) + TINY["f32"], c.what + " dgamma")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,C", SIZES + [(5000, 24), (3000, 640)])
def test_backward(M, C, dtype):
    c = Case(M, C, dtype, residual=False, gamma=C % 5 != 0)
    c.forward()
    check_backward(c, dh=M % 2 == 1, dgamma=C % 7 != 0)


@pytest.mark.parametrize("over", ["dy", "dh", "h"])
def test_backward_over_its_inputs(over):
    for M, C in [(3, 1000), (1100, 72), (2, 16384)]:
        c = Case(M, C, "bf16")
        c.forward()
        check_backward(c, over=over)


def test_backward_against_differences():
    """fp32 gradients of sum(y dy) along a direction against central differences of the fp64 definition."""
    c = Case(6, 50, "f32", residual=True)
    c.forward()
    rng = np.random.default_rng(1)
    dy, v = rng.standard_normal((2, 6, 50))
    u, t = rng.standard_normal(50), 1e-4
    dyd, dx, dg = torch.from_numpy(dy.astype(np.float32)).cuda(), torch.empty(6, 50, device="cuda"), torch.empty(50, device="cuda")
    n = c2.conv2d_rms_norm_bwd_workspace_bytes(6, 50)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    c2.conv2d_rms_norm_bwd(dyd, None, c.h, c.gamma, c.rstd, dx, dg, ws, n, 6, 50, 50, 0, c.h.ld, 50, c2.F32)
    x, r, g = c.x.host(), c.r.host(), c.gamma.double().cpu().numpy()
    f = lambda x, r, g: (ref.rms_norm(x, r, g, EPS)[1] * dy).sum()  # noqa: E731
    dx, dg = dx.double().cpu().numpy(), dg.double().cpu().numpy()
    # t^2 times third derivatives of order one, fp32 values off by some u of order 10
    for got, lo, hi in [((dx * v).sum(), (x - t * v, r, g), (x + t * v, r, g)),
                        ((dx * v).sum(), (x, r - t * v, g), (x, r + t * v, g)),
                        ((dg * u).sum(), (x, r, g - t * u), (x, r, g + t * u))]:
        assert abs(got - (f(*hi) - f(*lo)) / (2 * t)) < 1e-4


def test_a_second_call_on_another_stream_and_in_a_graph():
    """The same bits each time; every replay on new inputs against the eager call."""
    c = Case(300, 1000, "bf16")
    dy = Rows(300, 1000, "bf16", c.rng.standard_normal((300, 1000)))
    dg = torch.empty(1000, device="cuda")
    n = c2.conv2d_rms_norm_bwd_workspace_bytes(300, 1000)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    q, s = Rows(300, 1000, torch.int8), torch.empty(300, device="cuda")

    def step(stream=None):
        c.forward(stream)
        c2.conv2d_rms_norm_quant(c.x, c.r, c.gamma, None, q, s, None, 300, 1000, *c.ld("x", "r"), 0, q.ld, EPS, c2.BF16, stream)
        c2.conv2d_rms_norm_bwd(dy, None, c.h, c.gamma, c.rstd, c.dx, dg, ws, n, 300, 1000, dy.ld, 0, c.h.ld, c.dx.ld, c2.BF16,
                               stream)

    outs = lambda: [t.clone() for t in (c.h.store, c.y.store, c.rstd, q.store, s, c.dx.store, dg)]  # noqa: E731
    step()
    want = outs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    for a, b in zip(outs(), want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    for _ in range(3):
        c.x.view.normal_(generator=gen)
        graph.replay()
        torch.cuda.synchronize()
        got = outs()
        c.check()
        step()
        for a, b in zip(got, outs()):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Rows 2^22 elements apart: the last starts past 2^32 bytes."""
    M, C, ld = 600, 200, 1 << 22
    rng = np.random.default_rng(5)
    x = torch.zeros(M * ld, dtype=torch.bfloat16, device="cuda")
    x.view(M, ld)[:, :C].copy_(torch.from_numpy(rng.standard_normal((M, C))))
    host = x.view(M, ld)[:, :C].double().cpu().numpy()
    y, rstd = torch.empty(M, C, dtype=torch.bfloat16, device="cuda"), torch.empty(M, device="cuda")
    c2.conv2d_rms_norm(x, None, None, None, y, rstd, M, C, ld, 0, 0, C, EPS, c2.BF16)
    _, want, r = ref.rms_norm(host, None, None, EPS)
    inside(y.double().cpu().numpy(), want, (HALF["bf16"] + 30 * U) * np.abs(want), "far rows")
    dx = torch.empty(M, C, dtype=torch.bfloat16, device="cuda")
    c2.conv2d_rms_norm_bwd(y, None, x, None, rstd, dx, None, None, 0, M, C, C, 0, ld, C, c2.BF16)
    wdx, _ = ref.rms_norm_bwd(y.double().cpu().numpy(), None, host, None, rstd.cpu().numpy())
    inside(dx.double().cpu().numpy(), wdx, 2.0 ** -8 * np.abs(wdx) + 100 * U * r[:, None] * 4, "far rows dx")


def test_many_rows():
    """More rows than workgroups of a launch; a row each of one channel: y is gamma's sign of x, nearly."""
    M = (1 << 22) + 5
    x = torch.randn(M, 3, device="cuda").bfloat16()
    y, dg = torch.empty_like(x), torch.empty(3, device="cuda")
    rstd, dx = torch.empty(M, device="cuda"), torch.empty_like(x)
    c2.conv2d_rms_norm(x, None, None, None, y, rstd, M, 3, 3, 0, 0, 3, EPS, c2.BF16)
    v = x.double()
    r = (v.square().mean(1) + EPS).rsqrt()
    assert ((y.double() - v * r[:, None]).abs() <= (2.0 ** -8 + 30 * U) * (v * r[:, None]).abs() + 1e-37).all()
    n = c2.conv2d_rms_norm_bwd_workspace_bytes(M, 3)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    c2.conv2d_rms_norm_bwd(y, None, x, None, rstd, dx, dg, ws, n, M, 3, 3, 0, 3, 3, c2.BF16)
    terms = y.double() * v * rstd.double()[:, None]
    assert ((dg.double() - terms.sum(0)).abs() <= 772 * U * terms.abs().sum(0)).all()
