"""Rows in 8 bits and integer products on the GPU against the plain fp64
definitions (oracle/operators.py).

The sums are exact.  After them: the sum's conversion to fp32, the two scales'
product and the fused multiply-add round once each, so with u = 2^-24 a result
is off by at most 3 u of its terms' magnitudes, plus half a step of the output
type.  A quantised value lies within half a step and 3 u * 127 of 127 v / a
(the reciprocal, the product and, for the border, the reference's own value).
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

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = 1e-37


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


def tt(dtype):
    return torch.float32 if dtype == "f32" else torch.bfloat16


def lt(dtype):
    return c2.F32 if dtype == "f32" else c2.BF16


def rows(a, ld, skip, dtype, marker):
    """Device rows `ld` apart, `skip` elements into their storage; the rest holds a marker."""
    n, k = a.shape
    store = torch.full((skip + n * ld + 64,), marker, dtype=dtype, device="cuda")
    view = store[skip:skip + n * ld].view(n, ld)[:, :k]
    view.copy_(torch.as_tensor(a))
    return store, view


def untouched(store, n, k, ld, skip, marker):
    s = store.clone()
    s[skip:skip + n * ld].view(n, ld)[:, :k] = marker
    return bool((s == marker).all().item())


def inside(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = int(np.flatnonzero(bad.reshape(-1))[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; first {i}: got {got.reshape(-1)[i]!r} want "
                             f"{want.reshape(-1)[i]!r} tol {np.broadcast_to(tol, want.shape).reshape(-1)[i]!r}")


def run_product(M, K, N, dtype="bf16", bias=True, relu=False, padq=0, padw=0, pady=0, skip=0, seed=0, q=None, w=None,
                stream=None, check=True):
    rng = np.random.default_rng([seed, M, K, N])
    q = rng.integers(-128, 128, (M, K), dtype=np.int8) if q is None else q
    w = rng.integers(-128, 128, (N, K), dtype=np.int8) if w is None else w
    qs = np.exp(rng.standard_normal(M)).astype(np.float32)
    ws = (np.exp(rng.standard_normal(N)) / K).astype(np.float32)
    b = (10 * rng.standard_normal(N)).astype(np.float32) if bias else None
    what = f"M={M} K={K} N={N} {dtype} bias={bias} relu={relu} pads {padq} {padw} {pady} skip {skip}"
    print("[int8 product] " + what, file=sys.stderr, flush=True)
    # what lies between the rows must not enter the sums: a marker of 127s
    _, qd = rows(q, K + padq, skip, torch.int8, 127)
    _, wd = rows(w, K + padw, skip, torch.int8, 127)
    ystore, yd = rows(np.zeros((M, N), np.float32), N + pady, skip, tt(dtype), 7.0)
    qsd, wsd = torch.from_numpy(qs).cuda(), torch.from_numpy(ws).cuda()
    bd = torch.from_numpy(b).cuda() if bias else None
    n = c2.conv2d_int8_matmul_workspace_bytes(M, K, N)
    wk = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    torch.cuda.synchronize()
    c2.conv2d_int8_matmul(qd, qsd, wd, wsd, bd, yd, wk, n, M, K, N, K + padq, K + padw, N + pady, lt(dtype),
                          (c2.EPI_BIAS if bias else 0) | (c2.EPI_RELU if relu else 0), stream)
    torch.cuda.synchronize()
    got = yd.float().cpu().numpy().astype(np.float64)
    if check:
        want, size = ref.int8_matmul(q, qs, w, ws, b, relu)
        inside(got, want, 3 * U * size + HALF[dtype] * (np.abs(want) + 3 * U * size) + TINY, what)
        assert untouched(ystore, M, N, N + pady, skip, 7.0), what + ": wrote outside y"
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M", [1, 3, 16, 17, 32, 33, 64, 65, 130, 257])
def test_rows_and_channels(M, dtype):
    for K, N in [(1, 1), (16, 16), (48, 17), (64, 1), (128, 64), (144, 65), (1040, 130), (2048, 33), (127, 100),
                 (1037, 66), (515, 257)]:
        run_product(M, K, N, dtype, bias=(K + M) % 2 == 0, relu=(N + M) % 3 == 0)


# strides and starts: aligned (the fast kernels), then every other residue
@pytest.mark.parametrize("M", [5, 40, 150])
@pytest.mark.parametrize("padq,padw,skip", [(16, 32, 16), (1, 0, 0), (0, 3, 0), (2, 2, 2), (0, 0, 1), (0, 0, 3),
                                            (5, 7, 4), (0, 0, 8)])
def test_strides_and_alignment(M, padq, padw, skip):
    run_product(M, 208, 72, padq=padq, padw=padw, pady=3, skip=skip)
    run_product(M, 77, 72, padq=padq, padw=padw, pady=8, skip=skip, dtype="f32")


@pytest.mark.parametrize("M,K,N", [(40, 8192, 64), (200, 8192, 64), (200, 8191, 70), (66, 4096, 1000), (1, 16384, 64),
                                   (1, 4099, 300)])
def test_long_rows_split(M, K, N):
    run_product(M, K, N, "f32")
    run_product(M, K, N, "bf16", relu=True)


# the large tiles: whole, and with ragged edges on every side
@pytest.mark.parametrize("M,K,N", [(2048, 192, 2048), (2051, 144, 2100), (2050, 141, 2049), (4096, 256, 4096),
                                   (4100, 144, 4104), (4101, 400, 4099), (8192, 64, 2056), (4100, 512, 4104),
                                   (4100, 640, 4104)])
def test_large_tiles(M, K, N):
    for dtype in ("bf16", "f32"):
        run_product(M, K, N, dtype)


# many short rows: the weights stay in registers and the rows stream past, in
# every combination of k (up to 64, 128, 256, 512) and channels (up to 64, 128,
# 256, more), with tiles and channels that end inside a block
@pytest.mark.parametrize("K", [16, 64, 80, 128, 192, 256, 336, 512])
def test_short_rows_stream(K):
    for M, N in [(40001, 24), (33000, 64), (20011, 72), (16500, 128), (9001, 136), (9000, 256), (5003, 520)]:
        run_product(M, K, N, "bf16", bias=M % 2 == 0, relu=N % 3 == 0)
    for M, N in [(40001, 60), (20011, 100), (9001, 252), (5003, 516)]:
        run_product(M, K, N, "f32", padq=16, pady=4, bias=M % 2 == 1)


@pytest.mark.parametrize("M", [1, 64, 70])
def test_extreme_sums_are_exact(M):
    """-128 * -128 over the longest row: 2147467264, just below 2^31."""
    K, N = 131071, 20
    q = np.full((M, K), -128, np.int8)
    w = np.full((N, K), -128, np.int8)
    w[1::2] = 127
    run_product(M, K, N, "f32", bias=False, q=q, w=w)
    q = np.full((M, 131056), -128, np.int8)
    run_product(M, 131056, N, "f32", bias=False, q=q, w=w[:, :131056])


def test_repeatable_on_another_stream_and_in_a_graph():
    for M, K, N in [(4, 2048, 256), (200, 8192, 64), (300, 1001, 130), (4096, 128, 4096)]:
        a = run_product(M, K, N)
        st = torch.cuda.Stream()
        np.testing.assert_array_equal(a, run_product(M, K, N, stream=st, check=False))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    M, K, N = 200, 8192, 64
    x = torch.randn(M, K, generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.randint(-127, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    ws = torch.rand(N, generator=gen, device="cuda")
    q, qs = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    y = torch.empty(M, N, device="cuda")
    n = c2.conv2d_int8_matmul_workspace_bytes(M, K, N)
    wk = torch.empty(n, dtype=torch.uint8, device="cuda")

    def step():
        c2.conv2d_quantize_rows(x, q, qs, M, K, K, K, c2.BF16)
        c2.conv2d_int8_matmul(q, qs, w, ws, None, y, wk, n, M, K, N, K, K, N, c2.F32, 0)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (q, qs, y)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (q, qs, y):
            t.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((q, qs, y), want):
            assert torch.equal(a, b)


def test_scales_that_are_not_finite_show():
    """ReLU does not hide a NaN, and it stays in its row or channel."""
    for M in (5, 200):
        K, N = 64, 40
        q = torch.ones(M, K, dtype=torch.int8, device="cuda")
        w = torch.ones(N, K, dtype=torch.int8, device="cuda")
        qs, ws = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
        qs[2] = float("nan")
        ws[7] = float("nan")
        y = torch.zeros(M, N, device="cuda")
        n = c2.conv2d_int8_matmul_workspace_bytes(M, K, N)
        wk = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        c2.conv2d_int8_matmul(q, qs, w, ws, None, y, wk, n, M, K, N, K, K, N, c2.F32, c2.EPI_RELU)
        bad = torch.zeros(M, N, dtype=torch.bool)
        bad[2] = True
        bad[:, 7] = True
        assert torch.equal(torch.isnan(y).cpu(), bad)
        assert bool((y.cpu()[~bad] == 64.0).all())


# ------------------------------------------------------------------ rows in 8 bits

def run_rows(v, dtype, ldx=None, ldq=None, skip=0):
    M, K = v.shape
    ldx, ldq = ldx or K, ldq or K
    print(f"[rows] {M}x{K} {dtype} ld {ldx} {ldq} skip {skip}", file=sys.stderr, flush=True)
    _, xd = rows(v.astype(np.float32), ldx, skip, tt(dtype), 1e9)   # larger than any value
    qstore, qd = rows(np.zeros((M, K), np.int8), ldq, skip, torch.int8, 77)
    s = torch.full((M,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    c2.conv2d_quantize_rows(xd, qd, s, M, K, ldx, ldq, lt(dtype))
    torch.cuda.synchronize()
    assert untouched(qstore, M, K, ldq, skip, 77), "wrote outside q"
    return xd.float().cpu().numpy(), qd.cpu().numpy(), s.cpu().numpy()


def check_rows(x, q, s, what):
    t, scale = ref.quantise_rows(x)
    inside(s.astype(np.float64), scale, 2 * U * scale, what + " scale")
    inside(q.astype(np.float64), t, 0.5 + 3 * U * 127, what)
    assert np.abs(q.astype(np.int32)).max() <= 127


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 16), (100, 64), (33, 256), (2, 1000), (70, 1001), (9, 2048),
                                 (4, 4096), (3, 8192), (2, 20000), (2, 20001), (1000, 144), (3, 513)])
def test_quantize_rows(M, K, dtype):
    rng = np.random.default_rng([M, K])
    v = rng.standard_normal((M, K)) * np.exp(3 * rng.standard_normal((M, 1)))
    v[M // 2] *= 1e-30   # a tiny row
    if M > 2:
        v[1] = 0.0       # and an empty one
    check_rows(*run_rows(v, dtype), f"{M}x{K} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ldx,ldq,skip", [(64, 64, 0), (72, 80, 8), (68, 52, 4), (50, 50, 2), (49, 51, 1)])
def test_quantize_rows_strides(ldx, ldq, skip, dtype):
    v = np.random.default_rng(ldx).standard_normal((21, 48))
    check_rows(*run_rows(v, dtype, ldx, ldq, skip), f"ld {ldx} {ldq} skip {skip}")


def test_exact_grid_and_zero_rows():
    """Values on the grid come back exactly; a row of zeros has the floor's scale."""
    g = np.random.default_rng(0).integers(-127, 128, (16, 96)).astype(np.float64)
    g[:, 5] = 127
    g[3] = 0
    x, q, s = run_rows(g, "f32")
    np.testing.assert_array_equal(q, g.astype(np.int8))
    want = np.ones(16, np.float32)
    want[3] = np.float32(2.0 ** -100) / np.float32(127)
    np.testing.assert_array_equal(s, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [48, 49, 5000])
def test_rows_that_are_not_finite(K, dtype):
    v = np.random.default_rng(1).standard_normal((6, K))
    v[1, 3] = np.nan
    v[2, K - 1] = np.inf
    v[4, 0] = -np.inf
    x, q, s = run_rows(v, dtype)
    assert (np.isnan(s) == np.array([0, 1, 1, 0, 1, 0], bool)).all()
    assert (q[[1, 2, 4]] == 0).all()
    check_rows(x[[0, 3, 5]], q[[0, 3, 5]], s[[0, 3, 5]], "finite rows beside")


def test_offsets_past_32_bits():
    """Rows 2^21 bytes apart: the last starts past 2^32 bytes."""
    M, K, N, ld = 2100, 64, 48, 1 << 21
    rng = np.random.default_rng(2)
    q = rng.integers(-127, 128, (M, K), dtype=np.int8)
    w = rng.integers(-127, 128, (N, K), dtype=np.int8)
    store = torch.empty(M * ld, dtype=torch.int8, device="cuda")
    store.view(M, ld)[:, :K].copy_(torch.from_numpy(q))
    wd = torch.from_numpy(w).cuda()
    one = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    y = torch.empty(M, N, device="cuda")
    n = c2.conv2d_int8_matmul_workspace_bytes(M, K, N)
    wk = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    c2.conv2d_int8_matmul(store, one[0], wd, one[1], None, y, wk, n, M, K, N, ld, K, N, c2.F32, 0)
    np.testing.assert_array_equal(y.cpu().numpy(), (q.astype(np.int64) @ w.astype(np.int64).T).astype(np.float32))


def test_norm_quantised_then_product():
    """The whole path of a pre-activation 1x1 layer against fp64: the step of
    the 8-bit rows is the only error that counts."""
    N, C, H, W, G, K = 2, 128, 14, 15, 32, 72
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    x = torch.randn(N, H, W, C, generator=gen, device="cuda").to(torch.bfloat16)
    gamma = 1 + 0.2 * torch.randn(C, generator=gen, device="cuda")
    beta = 0.2 * torch.randn(C, generator=gen, device="cuda")
    wf = torch.randn(K, C, generator=gen, device="cuda")
    w, ws = torch.empty(K, C, dtype=torch.int8, device="cuda"), torch.empty(K, device="cuda")
    c2.conv2d_quantize_rows(wf, w, ws, K, C, C, C, c2.F32)
    M = N * H * W
    q, qs = torch.empty(M, C, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    y = torch.empty(M, K, device="cuda")
    n = max(c2.conv2d_group_norm_workspace_bytes(N, C, H, W, G), c2.conv2d_int8_matmul_workspace_bytes(M, C, K))
    wk = torch.empty(n, dtype=torch.uint8, device="cuda")
    c2.conv2d_group_norm_quant_nhwc(x, gamma, beta, q, qs, None, None, wk, n, N, C, H, W, G, C, C, 1e-5, c2.BF16,
                                    c2.ACT_SILU)
    c2.conv2d_int8_matmul(q, qs, w, ws, None, y, wk, n, M, C, K, C, C, K, c2.F32, 0)
    h, _, _ = ref.group_norm(x.float().cpu().numpy().astype(np.float64).reshape(N, H * W, C), gamma.cpu().numpy(),
                             beta.cpu().numpy(), G, 1e-5, ref.ACT_SILU)
    wq = w.cpu().numpy().astype(np.float64) * ws.cpu().numpy().astype(np.float64)[:, None]
    want = h.reshape(M, C) @ wq.T
    # half a step of every quantised value, with 1% for its own arithmetic
    _, scale = ref.quantise_rows(h.reshape(M, C))
    tol = 0.505 * scale[:, None] * np.abs(wq).sum(axis=1)
    inside(y.cpu().numpy().astype(np.float64), want, tol, "norm + product")
