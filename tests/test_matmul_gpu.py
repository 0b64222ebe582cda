"""Products with an epilogue and their gradients on the GPU against the plain
fp64 definitions (oracle/operators.py).

With u = 2^-24: a sum of K products (exact for bf16) is off by at most 2 K u of the
sum of its terms' magnitudes in whatever order, the bias adds one rounding.  An
activation's slope is at most 1.13, and its own arithmetic is off by (|z| + 10) u of
its value (SiLU: the exponent's rounding counts |z| times) or (2 z^2 + 16) u (GELU: the
complement of erf's argument counts z^2 times); the residual and the output round once
each.  Whole-number inputs whose sums stay below 2^24 have no rounding before the
output's.  The gradients' bf16 products see dz rounded to bf16: half a step of each term.
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
    from row_helpers import HALF, TINY, U, Rows, inside

ACTS = [0, 1, 2, 3]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


def lt(dtype):
    return c2.F32 if dtype == "f32" else c2.BF16


def whole(rng, shape):
    return rng.integers(-3, 4, shape).astype(np.float64)


def act_error(z, act):
    """Of the activation's own arithmetic, relative."""
    return {2: (np.abs(z) + 10) * U, 3: (2 * z * z + 16) * U}.get(act, 0.0)


def workspace(n, dtype="cuda"):
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None


def run_forward(M, K, N, dtype="bf16", bias=True, residual=True, z=True, act=0, padx=0, padw=0, pad=0, skip=0, ints=False,
                over=False, seed=0, stream=None):
    rng = np.random.default_rng([seed, M, K, N])
    make = whole if ints else lambda r, s: r.standard_normal(s)
    what = f"M={M} K={K} N={N} {dtype} bias={bias} res={residual} z={z} act={act} pads {padx} {padw} {pad} skip {skip} ints={ints}"
    print("[product] " + what, file=sys.stderr, flush=True)
    # what lies between the rows must not enter the sums
    x = Rows(M, K, dtype, make(rng, (M, K)), padx, skip, marker=float("nan"))
    w = Rows(N, K, dtype, make(rng, (N, K)), padw, skip, marker=float("nan"))
    b = torch.from_numpy(make(rng, N).astype(np.float32)).cuda() if bias else None
    r = Rows(M, N, dtype, make(rng, (M, N)), pad, skip) if residual else None
    zd = Rows(M, N, dtype, None, 2 * pad, skip) if z else None
    y = r if over else Rows(M, N, dtype, None, pad, skip)
    rh = r.host() if residual else None
    bh = b.cpu().numpy() if bias else None
    n = c2.conv2d_matmul_workspace_bytes(M, K, N, lt(dtype))
    ws = workspace(n)
    torch.cuda.synchronize()
    c2.conv2d_matmul(x, w, b, r, zd, y, ws, n, M, K, N, x.ld, w.ld, r.ld if residual else 0, zd.ld if z else 0, y.ld,
                     lt(dtype), act, stream)
    torch.cuda.synchronize()
    want, wz = ref.matmul(x.host(), w.host(), bh, rh, act)
    size = np.abs(x.host()) @ np.abs(w.host()).T + (np.abs(bh) if bias else 0)
    off = (0 if ints else 1) * (2 * K + 2) * U * size
    half = HALF[dtype]
    if z:
        inside(zd.host(), wz, off + half * (np.abs(wz) + off) + TINY[dtype], what + " z")
        assert zd.untouched(), what + ": wrote beside z"
    a = want - rh if residual else want
    off = 1.13 * off + act_error(wz, act) * np.abs(a) + (0 if ints and act < 2 else 2 * U * (np.abs(a) + np.abs(want)))
    inside(y.host(), want, off + half * (np.abs(want) + off) + TINY[dtype], what + " y")
    assert y.untouched(), what + ": wrote beside y"
    return y


SIZES = [(1, 1), (16, 16), (48, 17), (64, 1), (128, 64), (144, 65), (1040, 130), (2048, 33), (127, 100), (1037, 66),
         (515, 257), (8, 8)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 2, 3, 16, 17, 32, 33, 64, 65, 130, 257])
def test_rows_and_channels(M, dtype):
    for K, N in SIZES:
        run_forward(M, K, N, dtype, bias=(K + M) % 2 == 0, residual=(N + M) % 3 == 0, z=N % 2 == 0, act=(M + N) % 4)
        run_forward(M, K, N, dtype, bias=(K + M) % 2 == 1, residual=(N + M) % 3 == 1, z=N % 2 == 1, act=M % 2, ints=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 5, 40, 150])
@pytest.mark.parametrize("padx,padw,pad,skip", [(16, 32, 8, 16), (8, 0, 0, 8), (1, 0, 3, 0), (0, 3, 1, 0), (2, 2, 4, 2),
                                                (0, 0, 0, 1), (5, 7, 2, 4)])
def test_strides_and_alignment(M, padx, padw, pad, skip, dtype):
    for K in (208, 77):
        run_forward(M, K, 72, dtype, act=2, padx=padx, padw=padw, pad=pad, skip=skip)
        run_forward(M, K, 70, dtype, padx=padx, padw=padw, pad=pad, skip=skip, ints=True)


@pytest.mark.parametrize("M,K,N", [(40, 8192, 64), (200, 8192, 64), (200, 8191, 70), (66, 4096, 1000), (1, 16384, 64),
                                   (1, 4099, 300), (7, 4096, 4100)])
def test_long_sums(M, K, N):
    for dtype in ("f32", "bf16"):
        run_forward(M, K, N, dtype, act=3)
        run_forward(M, K, N, dtype, ints=True, act=1)


@pytest.mark.parametrize("M,K,N", [(2048, 192, 2048), (2051, 144, 2100), (2050, 141, 2049), (4096, 256, 4096),
                                   (4101, 400, 4099), (4100, 64, 2056), (20000, 64, 136), (70000, 24, 64)])
def test_large_tiles(M, K, N):
    for dtype in ("bf16", "f32"):
        run_forward(M, K, N, dtype, ints=True, act=1, z=False)
    run_forward(M, K, N, "bf16", act=2)


# rows of no whole number of 16-byte pieces, large enough to be copied first
@pytest.mark.parametrize("M,K,N,dtype", [(2051, 1037, 2100, "bf16"), (2049, 2047, 1030, "bf16"), (801, 1001, 700, "f32")])
def test_copied_operands(M, K, N, dtype):
    run_forward(M, K, N, dtype, act=2)
    run_forward(M, K, N, dtype, ints=True, act=1, padx=3, padw=1, pad=2, skip=1)
    run_backward(M, K, N, dtype, act=2)
    run_backward(M, K, N, dtype, act=0, ints=True, padx=3, padw=1, pad=2, skip=1)
    run_backward(M, K, N + 1, dtype, act=0, ints=True)
    run_backward(M, K, N, dtype, act=1, ints=True, want=("dx",))
    run_backward(M, K, N, dtype, act=1, ints=True, want=("dw", "db"))


@pytest.mark.parametrize("M", [1, 50, 300])
def test_y_over_the_residual(M):
    for dtype in ("bf16", "f32"):
        run_forward(M, 136, 72, dtype, act=2, over=True)
        run_forward(M, 4096, 72, dtype, over=True, pad=3, ints=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 70])
def test_activations_over_their_range(M, act):
    """x = z for one-column identities: every z from -30 to 30, and values that are not finite."""
    z = np.concatenate([np.linspace(-30, 30, 2001), [0.0, -0.0, 1e-30, -1e-30]]).astype(np.float32)
    w = torch.from_numpy(z[:, None].copy()).cuda()
    x = torch.ones(M, 1, device="cuda")
    y, zd = torch.empty(M, len(z), device="cuda"), torch.empty(M, len(z), device="cuda")
    n = c2.conv2d_matmul_workspace_bytes(M, 1, len(z), c2.F32)
    c2.conv2d_matmul(x, w, None, None, zd, y, workspace(n), n, M, 1, len(z), 1, 1, 0, len(z), len(z), c2.F32, act)
    want = ref.activate(z.astype(np.float64), act)
    inside(y.cpu().numpy(), np.broadcast_to(want, y.shape), (act_error(z.astype(np.float64), act) + U) * np.abs(want) + 1e-30,
           f"act {act}")
    np.testing.assert_array_equal(zd.cpu().numpy(), np.broadcast_to(z, y.shape))
    x[0] = float("nan")
    c2.conv2d_matmul(x, w, None, None, zd, y, workspace(n), n, M, 1, len(z), 1, 1, 0, len(z), len(z), c2.F32, act)
    assert torch.isnan(y[0]).all() and not torch.isnan(y[1:]).any()


# ------------------------------------------------------------------ gradients


def run_backward(M, K, N, dtype="bf16", act=0, want=("dx", "dw", "db"), padx=0, padw=0, pad=0, skip=0, ints=False, seed=0):
    rng = np.random.default_rng([seed, M, K, N])
    make = whole if ints else lambda r, s: r.standard_normal(s)
    what = f"M={M} K={K} N={N} {dtype} act={act} {want} pads {padx} {padw} {pad} skip {skip} ints={ints}"
    print("[gradients] " + what, file=sys.stderr, flush=True)
    nan = float("nan")
    x = Rows(M, K, dtype, make(rng, (M, K)), padx, skip, marker=nan)
    w = Rows(N, K, dtype, make(rng, (N, K)), padw, skip, marker=nan)
    dy = Rows(M, N, dtype, make(rng, (M, N)), pad, skip, marker=nan)
    z = Rows(M, N, dtype, make(rng, (M, N)), 2 * pad, skip, marker=nan) if act else None
    dx = Rows(M, K, dtype, None, pad, skip) if "dx" in want else None
    dw = Rows(N, K, dtype, None, 2 * pad, skip) if "dw" in want else None
    db = torch.full((N,), 7.0, device="cuda") if "db" in want else None
    n = c2.conv2d_matmul_bwd_workspace_bytes(M, K, N, lt(dtype))
    ws = workspace(n)
    torch.cuda.synchronize()
    c2.conv2d_matmul_bwd(dy, z, x, w, dx, dw, db, ws, n, M, K, N, dy.ld, z.ld if act else 0, x.ld, w.ld, dx.ld if dx else 0,
                         dw.ld if dw else 0, lt(dtype), act)
    torch.cuda.synchronize()
    zh = z.host() if act else None
    wx, ww, wb, dz = ref.matmul_bwd(dy.host(), zh, x.host(), w.host(), act)
    half = HALF[dtype]
    # dz: the slope's own arithmetic, and for bf16 the rounding that the products see
    slope = np.zeros_like(dz) if act < 2 else (act_error(zh, act) + 4 * U) * (1 + np.abs(zh)) * np.abs(dy.host())
    exact = ints and act < 2
    seen = slope + (0 if exact or dtype == "f32" or not act else half * (np.abs(dz) + slope))
    if dx:
        off = seen @ np.abs(w.host()) + (0 if exact else 1) * (2 * N + 2) * U * (np.abs(dz) @ np.abs(w.host()))
        inside(dx.host(), wx, off + half * (np.abs(wx) + off) + TINY[dtype], what + " dx")
        assert dx.untouched()
    if dw:
        off = seen.T @ np.abs(x.host()) + (0 if exact else 1) * (2 * M + 2) * U * (np.abs(dz).T @ np.abs(x.host()))
        inside(dw.host(), ww, off + half * (np.abs(ww) + off) + TINY[dtype], what + " dw")
        assert dw.untouched()
    if db is not None:
        off = slope.sum(axis=0) + (0 if exact else 1) * (min(M, 512) + 260) * U * np.abs(dz).sum(axis=0)
        inside(db.cpu().numpy(), wb, off + U * np.abs(wb) + TINY["f32"], what + " dbias")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 2, 7, 16, 33, 64, 65, 130, 257])
def test_gradients(M, dtype):
    for i, (K, N) in enumerate(SIZES):
        run_backward(M, K, N, dtype, act=(M + i) % 4)
        run_backward(M, K, N, dtype, act=i % 2, ints=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("padx,padw,pad,skip", [(16, 32, 8, 16), (8, 0, 0, 8), (1, 0, 3, 0), (0, 3, 1, 0), (2, 2, 4, 2),
                                                (0, 0, 0, 1), (5, 7, 2, 4)])
def test_gradients_strides_and_alignment(padx, padw, pad, skip, dtype):
    for M, K, N in [(5, 208, 72), (150, 77, 70), (150, 80, 64), (150, 77, 129)]:
        for act in (0, 2):
            run_backward(M, K, N, dtype, act=act, padx=padx, padw=padw, pad=pad, skip=skip)
        run_backward(M, K, N, dtype, act=1, padx=padx, padw=padw, pad=pad, skip=skip, ints=True)


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("db",), ("dx", "dw"), ("dw", "db"), ("dx", "db")])
@pytest.mark.parametrize("act", [0, 3])
def test_gradients_left_out(want, act):
    run_backward(100, 72, 136, act=act, want=want)
    run_backward(100, 73, 131, "f32", act=act, want=want)


@pytest.mark.parametrize("M,K,N", [(20000, 256, 64), (20003, 250, 61), (70001, 16, 24), (3, 300, 8192), (40, 64, 8191),
                                   (2048, 2048, 200), (2051, 2100, 144), (200, 2050, 2049), (4096, 4096, 128)])
def test_gradients_large(M, K, N):
    for dtype in ("bf16", "f32"):
        run_backward(M, K, N, dtype, act=1, ints=True)
    run_backward(M, K, N, "bf16", act=2)


def test_gradients_against_differences():
    """fp32 gradients of sum(y dy) along a direction against central differences of the fp64 definition."""
    rng = np.random.default_rng(2)
    M, K, N, t = 9, 20, 13, 1e-4
    x, w, b, r, dy = (rng.standard_normal(s).astype(np.float32) for s in ((M, K), (N, K), N, (M, N), (M, N)))
    for act in (0, 2, 3):
        d = [torch.from_numpy(v).cuda() for v in (x, w, b, r, dy)]
        y, z = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
        n = max(c2.conv2d_matmul_workspace_bytes(M, K, N, c2.F32), c2.conv2d_matmul_bwd_workspace_bytes(M, K, N, c2.F32))
        ws = workspace(n)
        c2.conv2d_matmul(d[0], d[1], d[2], d[3], z, y, ws, n, M, K, N, K, K, N, N, N, c2.F32, act)
        dx, dw, db = torch.empty(M, K, device="cuda"), torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
        c2.conv2d_matmul_bwd(d[4], z, d[0], d[1], dx, dw, db, ws, n, M, K, N, N, N, K, K, K, K, c2.F32, act)
        f = lambda x, w, b: (ref.matmul(x, w, b, r, act)[0] * dy).sum()  # noqa: E731
        for i, got in enumerate((dx, dw, db)):
            at = [v.astype(np.float64) for v in (x, w, b)]
            v = rng.standard_normal(at[i].shape)
            lo, hi = [list(at), list(at)]
            lo[i], hi[i] = at[i] - t * v, at[i] + t * v
            # t^2 of third derivatives of some hundred, fp32 sums off by some u of order 100
            assert abs((got.double().cpu().numpy() * v).sum() - (f(*hi) - f(*lo)) / (2 * t)) < 1e-3


def test_again_on_another_stream_and_in_a_graph():
    """The same bits each time; every replay on new inputs against the eager calls.  K and M are long enough to be split."""
    M, K, N = 200, 2048, 136
    rng = np.random.default_rng(4)
    put = lambda *s: torch.from_numpy(rng.standard_normal(s)).cuda().bfloat16()  # noqa: E731
    x, w, dy, b = put(M, K), put(N, K), put(M, N), torch.randn(N, device="cuda")
    z, y, dx, dw = put(M, N), put(M, N), put(M, K), put(N, K)
    db = torch.empty(N, device="cuda")
    n = max(c2.conv2d_matmul_workspace_bytes(M, K, N, c2.BF16), c2.conv2d_matmul_bwd_workspace_bytes(M, K, N, c2.BF16))
    ws = workspace(n)

    def step(stream=None):
        c2.conv2d_matmul(x, w, b, dy, z, y, ws, n, M, K, N, K, K, N, N, N, c2.BF16, 2, stream)
        c2.conv2d_matmul_bwd(dy, z, x, w, dx, dw, db, ws, n, M, K, N, N, N, K, K, K, K, c2.BF16, 2, stream)

    outs = lambda: [t.clone() for t in (z, y, dx, dw, db)]  # noqa: E731
    step()
    want = outs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    for a, c in zip(outs(), want):
        assert torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    for _ in range(3):
        x.normal_(generator=gen)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = outs()
        step()
        for a, c in zip(got, outs()):
            assert torch.equal(a, c)


def test_offsets_past_32_bits():
    """Rows 2^20 elements apart, the most that is taken: the last start past 2^32 bytes, in every operand's place."""
    M, K, N, ld = 2100, 40, 24, 1 << 20
    rng = np.random.default_rng(2)
    xh, wh, gh = whole(rng, (M, K)), whole(rng, (N, K)), whole(rng, (M, N))
    x = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda")
    x.view(M, ld)[:, :K].copy_(torch.from_numpy(xh))
    w, dy = torch.from_numpy(wh).cuda().bfloat16(), torch.from_numpy(gh).cuda().bfloat16()
    n = max(c2.conv2d_matmul_workspace_bytes(M, K, N, c2.BF16), c2.conv2d_matmul_bwd_workspace_bytes(M, K, N, c2.BF16))
    ws = workspace(n)
    y, dx, dw = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((M, N), (M, K), (N, K)))
    bf = lambda v: torch.from_numpy(v).bfloat16().double().numpy()  # noqa: E731
    c2.conv2d_matmul(x, w, None, None, None, y, ws, n, M, K, N, ld, K, 0, 0, N, c2.BF16, 0)
    np.testing.assert_array_equal(y.double().cpu().numpy(), bf(xh @ wh.T))
    c2.conv2d_matmul_bwd(dy, None, x, w, dx, dw, None, ws, n, M, K, N, N, 0, ld, K, K, K, c2.BF16, 0)
    np.testing.assert_array_equal(dw.double().cpu().numpy(), bf(gh.T @ xh))
    x.view(M, ld)[:, :N].copy_(dy)
    c2.conv2d_matmul_bwd(x, None, dx, w, y_dx := torch.empty_like(dx), None, None, ws, n, M, K, N, ld, 0, K, K, K, 0, c2.BF16, 0)
    np.testing.assert_array_equal(y_dx.double().cpu().numpy(), bf(gh @ wh))


def test_many_columns():
    """More columns than a launch of workgroups of 16 each has threads for."""
    N = (1 << 28) + 5
    w = torch.empty(N, dtype=torch.bfloat16, device="cuda").random_(-3, 4)
    x = torch.full((1, 1), 2.0, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(N, dtype=torch.bfloat16, device="cuda")
    n = c2.conv2d_matmul_workspace_bytes(1, 1, N, c2.BF16)
    c2.conv2d_matmul(x, w, None, None, None, y, workspace(n), n, 1, 1, N, 1, 1, 0, 0, N, c2.BF16, 0)
    assert torch.equal(y, 2 * w)
