"""Group norm with an activation (forward, quantised, backward) on the GPU
against the plain fp64 definitions (oracle/operators.py).

Tolerances, derived from the arithmetic (u = 2^-24, half a step of fp32):
a mean of fp32 sums is off by at most C u mean|x| with C = 64 (a thread's
run of values, then trees: fewer than 64 roundings reach any value), a
variance, and so rstd, by 64 u of itself; z by the errors of mean and rstd
and 4 u of its terms; the hardware's exp2 and reciprocal (1 ulp each) of an
argument rounded to u give a sigmoid within (2 |z| + 8) u; an output rounded
to its type adds half a step, eps / 2.
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
EPS = 1e-5
TINY = 1e-37  # below fp32's smallest normal magnitudes, which may be flushed


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


def tt(dtype):
    return torch.float32 if dtype == "f32" else torch.bfloat16


def lt(dtype):
    return c2.F32 if dtype == "f32" else c2.BF16


class Padded:
    """A [rows, cols] tensor with `ld` elements a row, starting `skip`
    elements into its storage; everything around it holds a marker."""

    def __init__(self, rows, cols, ld, skip, dtype, marker):
        self.rows, self.cols, self.ld, self.skip, self.marker = rows, cols, ld, skip, marker
        self.store = torch.full((skip + rows * ld + 64,), marker, dtype=dtype, device="cuda")
        self.view = self.store[skip:skip + rows * ld].view(rows, ld)[:, :cols]

    def untouched(self):
        s = self.store.clone()
        s[self.skip:self.skip + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = self.marker
        return bool((s == self.marker).all().item())


class Case:
    def __init__(self, N, C, H, W, G, act, dtype, pad=0, skip=0, offset=0.0, affine=True, seed=0):
        rng = np.random.default_rng([seed, N, C, H, W, G, act])
        self.N, self.C, self.H, self.W, self.G, self.act, self.dtype = N, C, H, W, G, act, dtype
        self.P, self.ld = H * W, C + pad
        t = tt(dtype)

        def put(a):
            p = Padded(N * self.P, C, self.ld, skip, t, 7.0)
            p.view.copy_(torch.from_numpy(a.reshape(N * self.P, C).astype(np.float32)))
            return p

        x = rng.standard_normal((N, self.P, C)) * np.exp(0.3 * rng.standard_normal(C)) + rng.standard_normal(C) + offset
        self.x = put(x)
        self.dy = put(rng.standard_normal((N, self.P, C)))
        self.affine = affine
        self.gamma = (1 + 0.2 * rng.standard_normal(C)).astype(np.float32) if affine else np.ones(C, np.float32)
        self.beta = (0.2 * rng.standard_normal(C)).astype(np.float32) if affine else np.zeros(C, np.float32)
        self.gd = torch.from_numpy(self.gamma).cuda() if affine else None
        self.bd = torch.from_numpy(self.beta).cuda() if affine else None
        self.y = Padded(N * self.P, C, self.ld, skip, t, 7.0)
        self.mean = torch.full((N, G), float("nan"), device="cuda")
        self.rstd = torch.full((N, G), float("nan"), device="cuda")

    def host(self, p):
        return p.view.float().cpu().numpy().astype(np.float64).reshape(self.N, self.P, self.C)

    def workspace(self, backward=False):
        n = c2.conv2d_group_norm_workspace_bytes(self.N, self.C, self.H, self.W, self.G, backward)
        assert n > 0
        return torch.full((n,), 255, dtype=torch.uint8, device="cuda"), n   # NaN bits: nothing relies on it

    def forward(self, stream=None):
        ws, n = self.workspace()
        c2.conv2d_group_norm_nhwc(self.x.view, self.gd, self.bd, self.y.view, self.mean, self.rstd, ws, n, self.N,
                                  self.C, self.H, self.W, self.G, self.ld, self.ld, EPS, lt(self.dtype), self.act,
                                  stream)

    # ---- reference values and their tolerances
    def errors(self, mean_exact=False):
        x = self.host(self.x)
        cg = self.C // self.G
        mean, rstd = ref.group_stats(x, self.G, EPS)
        per = lambda s: np.repeat(s, cg, axis=1)[:, None, :]  # noqa: E731
        e_mean = 64 * U * np.abs(x).reshape(self.N, self.P, self.G, cg).mean(axis=(1, 3)) + TINY
        # an error of the mean moves the variance by its square
        e_rstd = rstd * (64 * U + (e_mean * rstd) ** 2)
        xh = ref.normalise(x, mean, rstd)
        z = xh * self.gamma + self.beta
        e_z = (np.abs(self.gamma) * (per(rstd * e_mean) + np.abs(xh) * (per(e_rstd / rstd) + 4 * U)) +
               4 * U * (np.abs(z) + np.abs(self.beta)) + TINY)
        y = ref.activate(z, self.act)
        e_y = 1.1 * e_z + ((2 * np.abs(z) + 8) * U * np.abs(y) if self.act == ref.ACT_SILU else 0.0) + TINY
        return dict(x=x, mean=mean, rstd=rstd, e_mean=e_mean, e_rstd=e_rstd, xh=xh, z=z, e_z=e_z, y=y, e_y=e_y)


def inside(got, want, tol, what):
    got = np.asarray(got, np.float64)
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = int(np.flatnonzero(bad.reshape(-1))[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; first {i}: got {got.reshape(-1)[i]!r} want "
                             f"{np.broadcast_to(want, got.shape).reshape(-1)[i]!r} tol "
                             f"{np.broadcast_to(tol, got.shape).reshape(-1)[i]!r}")


def check_forward(c, what):
    e = c.errors()
    inside(c.mean.cpu().numpy(), e["mean"], e["e_mean"], what + " mean")
    inside(c.rstd.cpu().numpy(), e["rstd"], e["e_rstd"] + 2 * U * e["rstd"], what + " rstd")
    inside(c.host(c.y), e["y"], e["e_y"] + HALF[c.dtype] * (np.abs(e["y"]) + e["e_y"]), what + " y")
    assert c.y.untouched(), what + ": wrote outside y"


#        N  C     H    W    G
SIZES = [(1, 1, 1, 1, 1),          # one value: the variance is 0
         (2, 16, 1, 1, 4),         # one pixel
         (1, 6, 3, 5, 3),
         (2, 117, 7, 9, 9),        # odd channels, groups of 13
         (3, 144, 19, 13, 9),
         (1, 256, 28, 28, 32),
         (2, 2048, 5, 3, 32),
         (1, 4096, 3, 3, 1),       # the widest, one group
         (1, 4095, 2, 3, 65),
         (2, 1000, 9, 7, 1000),    # a group per channel
         (1, 8, 130, 121, 2),      # few channels, many pixels
         (70, 24, 6, 5, 1),        # many images
         (4, 32, 64, 63, 8)]
ACTS = [0, 1, 2]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, dtype):
    for act in ACTS:
        print(f"[group norm] {size} {dtype} act {act}", file=sys.stderr, flush=True)
        c = Case(*size, act, dtype)
        c.forward()
        check_forward(c, f"{size} {dtype} act {act}")


# row strides and starts that leave 16, 8, 4 or 2 bytes of alignment
LAYOUTS = [(8, 0), (4, 4), (2, 2), (1, 1), (16, 8)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,skip", LAYOUTS)
def test_forward_strides(pad, skip, dtype):
    c = Case(2, 48, 9, 11, 6, 2, dtype, pad=pad, skip=skip)
    c.forward()
    check_forward(c, f"pad {pad} skip {skip} {dtype}")


def test_forward_without_affine_and_stats():
    c = Case(2, 40, 9, 11, 5, 0, "bf16", affine=False)
    c.forward()
    check_forward(c, "no affine")
    saved = c.host(c.y)
    ws, n = c.workspace()
    c.y.view.fill_(0)
    c2.conv2d_group_norm_nhwc(c.x.view, None, None, c.y.view, None, None, ws, n, c.N, c.C, c.H, c.W, c.G, c.ld, c.ld,
                              EPS, c2.BF16, 0)
    np.testing.assert_array_equal(c.host(c.y), saved)


@pytest.mark.parametrize("offset", [1e3, -1e4])
def test_forward_far_from_zero(offset):
    """A mean of 1e3 to 1e4 standard deviations: no cancellation in the variance."""
    c = Case(2, 64, 33, 31, 8, 0, "f32", offset=offset)
    c.forward()
    check_forward(c, f"offset {offset}")


def test_forward_in_place_and_repeatable():
    c = Case(2, 96, 21, 23, 8, 2, "bf16")
    c.forward()
    first, mean = c.host(c.y), c.mean.clone()
    c.forward()
    np.testing.assert_array_equal(c.host(c.y), first)
    assert torch.equal(c.mean, mean)
    ws, n = c.workspace()
    c2.conv2d_group_norm_nhwc(c.x.view, c.gd, c.bd, c.x.view, None, None, ws, n, c.N, c.C, c.H, c.W, c.G, c.ld, c.ld,
                              EPS, c2.BF16, 2)
    np.testing.assert_array_equal(c.host(c.x), first)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_stay_in_their_group(bad):
    clean, c = (Case(2, 32, 13, 7, 4, 1, "f32") for _ in range(2))
    c.x.view[5, 9] = bad   # image 0, channel 9: group 1
    clean.forward()
    c.forward()
    a, b = clean.host(clean.y), c.host(c.y)
    assert np.isnan(b[0, :, 8:16]).all()
    a[0, :, 8:16] = b[0, :, 8:16] = 0
    np.testing.assert_array_equal(a, b)
    assert np.isnan(c.rstd.cpu().numpy()[0, 1])


def test_forward_on_another_stream_and_in_a_graph():
    c = Case(2, 64, 17, 19, 8, 2, "bf16")
    c.forward()
    want = c.host(c.y)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    c.y.view.fill_(0)
    torch.cuda.synchronize()
    c.forward(st)
    st.synchronize()
    np.testing.assert_array_equal(c.host(c.y), want)
    ws, n = c.workspace(True)
    dx = torch.empty_like(c.x.view)
    dg, db = torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    q = torch.empty(c.N * c.P, 64, dtype=torch.int8, device="cuda")
    qs = torch.empty(c.N * c.P, device="cuda")

    def step(stream=None):
        args = (ws, n, c.N, c.C, c.H, c.W, c.G)
        c2.conv2d_group_norm_nhwc(c.x.view, c.gd, c.bd, c.y.view, c.mean, c.rstd, *args, c.ld, c.ld, EPS, c2.BF16, 2,
                                  stream)
        c2.conv2d_group_norm_bwd_nhwc(c.dy.view, c.x.view, c.gd, c.bd, c.mean, c.rstd, dx, dg, db, *args, c.ld, c.ld,
                                      64, c2.BF16, 2, stream)
        c2.conv2d_group_norm_quant_nhwc(c.x.view, c.gd, c.bd, q, qs, None, None, *args, c.ld, 64, EPS, c2.BF16, 2,
                                        stream)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (c.y.view, c.mean, c.rstd, dx, dg, db, q, qs)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (c.y.view, c.mean, c.rstd, dx, dg, db, q, qs):
            t.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((c.y.view, c.mean, c.rstd, dx, dg, db, q, qs), want):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """4096 pixels 2^20 elements apart: element offsets up to 2^32."""
    N, C, H, W, G, ld = 1, 32, 64, 64, 4, 1 << 20
    x = torch.empty(H * W * ld, dtype=torch.bfloat16, device="cuda")
    view = x.view(H * W, ld)[:, :C]
    torch.manual_seed(1)
    view.copy_(torch.randn(H * W, C))
    dense = view.contiguous()
    y, y2 = torch.empty_like(dense), torch.empty_like(dense)
    n = c2.conv2d_group_norm_workspace_bytes(N, C, H, W, G)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    c2.conv2d_group_norm_nhwc(dense, None, None, y, None, None, ws, n, N, C, H, W, G, C, C, EPS, c2.BF16, 2)
    c2.conv2d_group_norm_nhwc(x, None, None, y2, None, None, ws, n, N, C, H, W, G, ld, C, EPS, c2.BF16, 2)
    assert torch.equal(y, y2)
    c2.conv2d_group_norm_nhwc(dense, None, None, x, None, None, ws, n, N, C, H, W, G, C, ld, EPS, c2.BF16, 2)
    assert torch.equal(view, y)


# ------------------------------------------------------------------ quantised

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_quantised(size, dtype):
    for act in ACTS:
        print(f"[group norm quant] {size} {dtype} act {act}", file=sys.stderr, flush=True)
        c = Case(*size, act, dtype)
        ws, n = c.workspace()
        q = Padded(c.N * c.P, c.C, c.C + 3, 5, torch.int8, 77)
        s = torch.full((c.N * c.P,), float("nan"), device="cuda")
        c2.conv2d_group_norm_quant_nhwc(c.x.view, c.gd, c.bd, q.view, s, c.mean, c.rstd, ws, n, c.N, c.C, c.H, c.W,
                                        c.G, c.ld, c.C + 3, EPS, lt(dtype), act)
        check_quantised(c, q, s, f"{size} {dtype} act {act}")


def check_quantised(c, q, s, what):
    e = c.errors()
    inside(c.mean.cpu().numpy(), e["mean"], e["e_mean"], what + " mean")
    y = e["y"].reshape(-1, c.C)
    e_y = e["e_y"].reshape(-1, c.C)
    t, scale = ref.quantise_rows(y)
    e_top = e_y.max(axis=1)
    a = scale * 127.0
    inside(s.cpu().numpy(), scale, e_top / 127.0 + 4 * U * scale, what + " scale")
    # half a step, and what the errors of the value and of the row's maximum move
    tol = 0.5 + (127.0 / a)[:, None] * e_y + np.abs(t) * (e_top / a + 4 * U)[:, None] + 127 * 4 * U
    inside(q.view.cpu().numpy(), t, tol, what + " q")
    assert q.untouched(), what + ": wrote outside q"


@pytest.mark.parametrize("ldq", [48, 64, 56, 52, 50, 49])
def test_quantised_strides(ldq):
    c = Case(2, 48, 9, 11, 6, 2, "bf16")
    ws, n = c.workspace()
    q = Padded(c.N * c.P, 48, ldq, 0, torch.int8, 77)
    s = torch.empty(c.N * c.P, device="cuda")
    c2.conv2d_group_norm_quant_nhwc(c.x.view, c.gd, c.bd, q.view, s, c.mean, c.rstd, ws, n, c.N, c.C, c.H, c.W, c.G,
                                    c.ld, ldq, EPS, c2.BF16, 2)
    check_quantised(c, q, s, f"ldq {ldq}")


# ------------------------------------------------------------------ backward

def backward(c, want_params=True, dx=None):
    ws, n = c.workspace(True)
    dx = dx or c.y
    dg = torch.full((c.C,), float("nan"), device="cuda") if want_params else None
    db = torch.full((c.C,), float("nan"), device="cuda") if want_params else None
    c2.conv2d_group_norm_bwd_nhwc(c.dy.view, c.x.view, c.gd, c.bd, c.mean, c.rstd, dx.view, dg, db, ws, n, c.N, c.C,
                                  c.H, c.W, c.G, c.ld, c.ld, c.ld, lt(c.dtype), c.act)
    return dg, db


def check_backward(c, dg, db, what, dx=None):
    x, dy = c.host(c.x), c.host(c.dy)
    mean, rstd = (t.cpu().numpy().astype(np.float64) for t in (c.mean, c.rstd))
    wdx, wdg, wdb = ref.group_norm_bwd(dy, x, c.gamma, c.beta, mean, rstd, c.act)
    cg = c.C // c.G
    per = lambda s: np.repeat(s, cg, axis=1)[:, None, :]  # noqa: E731
    grp = lambda t: t.reshape(c.N, c.P, c.G, cg).mean(axis=(1, 3))  # noqa: E731
    xh = ref.normalise(x, mean, rstd)
    z = xh * c.gamma + c.beta
    dz = dy * ref.activation_slope(z, c.act)
    e_z = 4 * U * (np.abs(xh * c.gamma) + np.abs(c.beta))
    if c.act == ref.ACT_RELU:
        e_dz = np.where(np.abs(z) <= e_z, np.abs(dy), 0.0)   # the border may fall on either side
    elif c.act == ref.ACT_SILU:
        # the slope's own slope is below 1/2; its terms come from a sigmoid within (2 |z| + 8) u
        e_dz = np.abs(dy) * (0.5 * e_z + (1 + np.abs(z)) * (2 * np.abs(z) + 8 + 4) * U * ref.sigmoid(z) + 4 * U)
    else:
        e_dz = 0.0 * dy
    ag = np.abs(c.gamma)
    inside(db.cpu().numpy(), wdb, e_dz.sum(axis=(0, 1)) + 64 * U * np.abs(dz).sum(axis=(0, 1)) + TINY, what + " dbeta")
    inside(dg.cpu().numpy(), wdg, (e_dz * np.abs(xh)).sum(axis=(0, 1)) +
           68 * U * np.abs(dz * xh).sum(axis=(0, 1)) + TINY, what + " dgamma")
    e_s1 = grp(ag * e_dz + 68 * U * ag * np.abs(dz))
    e_s2 = grp((ag * e_dz + 72 * U * ag * np.abs(dz)) * np.abs(xh))
    s1, s2 = np.abs(grp(c.gamma * dz)), np.abs(grp(c.gamma * dz * xh))
    e_dx = per(np.abs(rstd)) * (ag * e_dz + per(e_s1) + np.abs(xh) * per(e_s2) +
                                8 * U * (ag * np.abs(dz) + per(s1) + np.abs(xh) * per(s2))) + TINY
    got = c.host(dx or c.y)
    inside(got, wdx, e_dx + HALF[c.dtype] * (np.abs(wdx) + e_dx), what + " dx")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(size, dtype):
    for act in ACTS:
        print(f"[group norm backward] {size} {dtype} act {act}", file=sys.stderr, flush=True)
        c = Case(*size, act, dtype)
        c.forward()
        dg, db = backward(c)
        check_backward(c, dg, db, f"{size} {dtype} act {act}")
        assert c.y.untouched(), "wrote outside dx"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,skip", LAYOUTS)
def test_backward_strides(pad, skip, dtype):
    c = Case(2, 48, 9, 11, 6, 2, dtype, pad=pad, skip=skip)
    c.forward()
    dg, db = backward(c)
    check_backward(c, dg, db, f"pad {pad} skip {skip} {dtype}")
    assert c.y.untouched()


def test_backward_options():
    """No affine, no parameter gradients, dx over dy; equal calls, equal bits."""
    c = Case(3, 40, 9, 11, 5, 1, "bf16", affine=False)
    c.forward()
    dg, db = backward(c)
    check_backward(c, dg, db, "no affine")
    first = c.host(c.y)
    dg2, db2 = backward(c)
    assert torch.equal(dg, dg2) and torch.equal(db, db2)
    backward(c, want_params=False, dx=c.dy)
    np.testing.assert_array_equal(c.host(c.dy), first)


def test_backward_against_differences():
    """Directional differences of the fp64 forward through the kernel's
    gradients: sum(dx * v) against (f(x + h v) - f(x - h v)) / 2h."""
    c = Case(2, 24, 5, 7, 3, 2, "f32")
    c.forward()
    dg, db = backward(c)
    x, dy = c.host(c.x), c.host(c.dy)
    gamma, beta = c.gamma.astype(np.float64), c.beta.astype(np.float64)
    f = lambda x, g, b: float((ref.group_norm(x, g, b, c.G, EPS, c.act)[0] * dy).sum())  # noqa: E731
    rng = np.random.default_rng(3)
    h = 1e-5
    got = dict(x=c.host(c.y), g=dg.cpu().numpy().astype(np.float64), b=db.cpu().numpy().astype(np.float64))
    for name in ("x", "g", "b"):
        v = rng.standard_normal(got[name].shape)
        p = [dict(x=x, g=gamma, b=beta)[k] + (h * v if k == name else 0) for k in ("x", "g", "b")]
        m = [dict(x=x, g=gamma, b=beta)[k] - (h * v if k == name else 0) for k in ("x", "g", "b")]
        want = (f(*p) - f(*m)) / (2 * h)
        mine = float((got[name] * v).sum())
        # fp32 gradients: 200 u of the terms' magnitudes; the differences: h^2
        assert abs(mine - want) <= 200 * U * float(np.abs(got[name] * v).sum()) + 1e-6, (name, mine, want)
