"""Operators at sizes that one launch or one 32-bit grid does not hold: every
result compared on the device, part by part, with values made so that the
answers are exact.
"""
import sys

import pytest

from helpers import ensure_built, gpu_available

pytestmark = pytest.mark.gpu

if gpu_available():
    ensure_built()
    import torch
    import cnn_convolution_conv2d_amd as c2

TOP = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def say(*what):
    print("[large sizes]", *what, file=sys.stderr, flush=True)


def parts(n, each):
    return ((i, min(i + each, n)) for i in range(0, n, each))


@pytest.mark.parametrize("M,K", [(TOP, 16), (TOP - 200, 17)])   # rows that stream past the weights; unaligned rows
def test_product_of_as_many_rows_as_an_int_holds(M, K):
    """Integer sums below 2^24 and scales that are powers of two: fp32 results are exact."""
    say("product", M, K)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(K)
    q = torch.empty(M, K, dtype=torch.int8, device="cuda")
    qs = torch.empty(M, device="cuda")
    for a, b in parts(M, 1 << 27):
        q[a:b].random_(-128, 128, generator=gen)
        qs[a:b] = torch.exp2(torch.randint(-3, 4, (b - a,), generator=gen, device="cuda").float())
    w = torch.randint(-128, 128, (1, K), generator=gen, device="cuda", dtype=torch.int8)
    y = torch.full((M + 64, 1), -77.5, device="cuda")
    c2.conv2d_int8_matmul(q, qs, w, torch.full((1,), 0.25, device="cuda"), None, y, None, 0, M, K, 1, K, K, 1, c2.F32, 0)
    torch.cuda.synchronize()
    for a, b in parts(M, 1 << 26):
        acc = torch.zeros(b - a, device="cuda")
        for k in range(K):
            acc += q[a:b, k].float() * float(w[0, k])
        assert torch.equal(y[a:b, 0], acc * qs[a:b] * 0.25), (a, b)
    assert bool((y[M:] == -77.5).all())


#                          lanes that share a row: 64, 4 vectors each; a workgroup
@pytest.mark.parametrize("M,K", [(2 ** 26 + 77, 520), (2 ** 24 + 33, 2050)])
def test_more_rows_in_8_bits_than_a_grid_holds(M, K):
    """Whole numbers up to 127, one of them in every row: the rows come back as they are, with scale 1."""
    say("rows", M, K)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(K)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    for a, b in parts(M, 1 << 22):
        x[a:b] = torch.randint(-126, 127, (b - a, K), generator=gen, device="cuda", dtype=torch.int8)
    x[:, K - 1] = 127
    q = torch.empty(M, K, dtype=torch.int8, device="cuda")
    s = torch.empty(M, device="cuda")
    c2.conv2d_quantize_rows(x, q, s, M, K, K, K, c2.BF16)
    torch.cuda.synchronize()
    for a, b in parts(M, 1 << 22):
        assert torch.equal(q[a:b].bfloat16(), x[a:b]), (a, b)
    assert bool((s == 1).all())


U, HALF, EPS = 2.0 ** -24, 2.0 ** -8, 1e-5

#             N           C   H  W   G
IMAGES = [(70000, 16, 7, 7, 2),          # more than 65535 images whose chunks exchange their sums
          (2 ** 24 + 3, 16, 1, 1, 2),    # the same form, in two launches
          (2 ** 24 + 5, 18, 1, 1, 9),    # a stream over memory
          (2 ** 20, 512, 1, 1, 16)]      # a group in registers: 2^24 of them


def within(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    if bool(bad.any()):
        i = int(bad.reshape(-1).nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} off; first {i}: got {float(got.reshape(-1)[i])!r} want "
                             f"{float(want.reshape(-1)[i])!r} tol {float(tol.expand_as(want).reshape(-1)[i])!r}")


@pytest.mark.parametrize("N,C,H,W,G", IMAGES)
def test_more_images_than_a_grid_holds(N, C, H, W, G):
    """Group norm forward, quantised and backward in bf16, with the bounds of the small
    sizes: 2 u of the largest magnitude for a mean, 8 u for rstd, 64 u for sums
    over an image's group, half a step of each output."""
    say("images", N, C, H, W, G)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(N)
    P, cg, M = H * W, C // G, N * H * W
    each = max(1, (1 << 25) // (P * C))   # images compared at a time
    x = torch.empty(N, P, C, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    dy = torch.empty_like(x).normal_(generator=gen)
    y, q = torch.empty_like(x), torch.empty(N, P, C, dtype=torch.int8, device="cuda")
    qs = torch.empty(N, P, device="cuda")
    mean, rstd = torch.empty(N, G, device="cuda"), torch.empty(N, G, device="cuda")
    dg, db = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    n = c2.conv2d_group_norm_workspace_bytes(N, C, H, W, G, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    size = (N, C, H, W, G)

    def expected(a, b):
        v = x[a:b].double().view(-1, P, G, cg)
        mu = v.mean((1, 3))
        var = (v - mu[:, None, :, None]).square().mean((1, 3))
        return v, mu, (var + EPS) ** -0.5, v.abs().amax((1, 3))

    c2.conv2d_group_norm_nhwc(x, None, None, y, mean, rstd, ws, n, *size, C, C, EPS, c2.BF16, 0)
    c2.conv2d_group_norm_quant_nhwc(x, None, None, q, qs, None, None, ws, n, *size, C, C, EPS, c2.BF16, 0)
    for a, b in parts(N, each):
        v, mu, r, top = expected(a, b)
        within(mean[a:b], mu, 2 * U * top, "mean")
        within(rstd[a:b], r, r * (8 * U + (2 * U * top * r) ** 2), "rstd")
        per = lambda s: s[:, None, :, None]  # noqa: E731
        xh = (v - per(mu)) * per(r)
        e = per(2 * U * top * r) + xh.abs() * (16 * U + per((2 * U * top * r) ** 2))
        within(y[a:b].view(v.shape), xh, e + HALF * (xh.abs() + e), "y")
        xh, e = xh.reshape(-1, P, C), e.reshape(-1, P, C)
        amax = xh.abs().amax(2, keepdim=True).clamp_min(2.0 ** -100)
        e_top = e.amax(2, keepdim=True)
        within(qs[a:b][..., None], amax / 127, e_top / 127 + 4 * U * amax / 127, "scale")
        within(q[a:b], xh * 127 / amax, 0.5 + 127 / amax * (e + xh.abs() * (e_top / amax + 4 * U)) + 512 * U, "q")
    del q, qs
    for want_params in (True, False):
        dx = y.zero_()
        c2.conv2d_group_norm_bwd_nhwc(dy, x, None, None, mean, rstd, dx, dg if want_params else None,
                                      db if want_params else None, ws, n, *size, C, C, C, c2.BF16, 0)
        gsum, bsum, gabs, babs = (torch.zeros(C, dtype=torch.float64, device="cuda") for _ in range(4))
        for a, b in parts(N, each):
            v, dz = x[a:b].double().view(-1, P, G, cg), dy[a:b].double().view(-1, P, G, cg)
            per = lambda s: s.double()[:, None, :, None]  # noqa: E731
            r = per(rstd[a:b])
            xh = (v - per(mean[a:b])) * r
            avg = lambda t: t.mean((1, 3), keepdim=True)  # noqa: E731
            want = r * (dz - avg(dz) - xh * avg(dz * xh))
            e = 80 * U * r * (dz.abs() + avg(dz.abs()) + xh.abs() * avg((dz * xh).abs()))
            within(dx[a:b].view(v.shape), want, e + HALF * (want.abs() + e), "dx")
            t = dz * xh
            for acc, add in ((gsum, t), (bsum, dz), (gabs, t.abs()), (babs, dz.abs())):
                acc += add.sum((0, 1)).reshape(C)
        if want_params:
            within(dg, gsum, 72 * U * gabs, "dgamma")
            within(db, bsum, 64 * U * babs, "dbeta")
