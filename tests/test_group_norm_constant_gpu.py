"""Group norm of groups that are constant, or nearly so and far from zero, where
1 / sqrt(var + eps) is large: forward and quantised, in every form.
"""
import sys

import numpy as np
import pytest

import test_group_norm_gpu as small
from helpers import gpu_available
from oracle import operators as ref
from test_group_norm_statistics_gpu import case, quantised

pytestmark = pytest.mark.gpu

U = small.U


@pytest.fixture(autouse=True)
def _need_gpu():
    if not gpu_available():
        pytest.skip("no GPU")


def say(*what):
    print("[constant groups]", *what, file=sys.stderr, flush=True)


#              N  C     H    W    G
CONSTANT = [(2, 32, 7, 7, 4),          # a group in registers; quantised in one launch
            (1, 2048, 16, 16, 2),      # two launches
            (2, 520, 13, 11, 65),      # and quantised with a wave per pixel
            (2, 128, 160, 165, 32),    # chunks that exchange their sums, the quantised pass too
            (2, 48, 30, 31, 6)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", CONSTANT, ids=str)
@pytest.mark.parametrize("value", [100.0, 1000.0, 1000.1])
def test_constant_groups_give_beta(size, dtype, value):
    """x - mean is 0 exactly, whatever 1 / sqrt(eps) multiplies it with."""
    for act in (0, 2):
        say(size, dtype, value, act)
        c = case(size, act, dtype, lambda x: x.fill_(value))
        c.forward()
        want = ref.activate(np.broadcast_to(c.beta.astype(np.float64), (c.N, c.P, c.C)), act)
        tol = 32 * U * np.abs(want) + small.TINY   # beta goes through; the sigmoid's arguments are below 2
        got = c.host(c.y)
        small.inside(got, want, tol + small.HALF[dtype] * (np.abs(want) + tol), "constant y")
        assert (c.mean.cpu() == c.x.view.flatten()[0].float().cpu()).all()
        q, s = quantised(c)
        t, scale = ref.quantise_rows(want.reshape(-1, c.C))
        small.inside(s.cpu().numpy(), scale, 40 * U * scale, "constant scale")
        small.inside(q.view.cpu().numpy(), t, 0.5 + 127 * 80 * U, "constant q")


def test_constant_groups_without_beta_quantise_to_zero():
    for size in CONSTANT:
        say(size, "no affine")
        c = small.Case(*size, 0, "bf16", affine=False)
        c.x.view.fill_(1000.0)
        q, _ = quantised(c)
        assert not bool(q.view.any())


@pytest.mark.parametrize("size", CONSTANT, ids=str)
@pytest.mark.parametrize("offset", [100.0, 1000.0, -30000.0])
def test_bf16_far_from_zero(size, offset):
    """Nearly constant: of the values around the offset bf16 keeps a step or a few.
    z is off by the mean's rounding (2 u of |mean|, times rstd gamma) and 8 u of
    its terms."""
    for act in (0, 2):
        say(size, "offset", offset, act)
        c = small.Case(*size, act, "bf16", offset=offset)
        c.forward()
        x = c.host(c.x)
        mean, rstd = ref.group_stats(x, c.G, small.EPS)
        per = lambda s: np.repeat(s, c.C // c.G, axis=1)[:, None, :]  # noqa: E731
        top = np.abs(x).reshape(c.N, c.P, c.G, -1).max(axis=(1, 3))
        e_mean, r = 2 * U * top, 8 * U + (2 * U * top * rstd) ** 2
        xh = ref.normalise(x, mean, rstd)
        z = xh * c.gamma + c.beta
        e_z = np.abs(c.gamma) * (per(rstd * e_mean) + np.abs(xh) * per(r)) + 8 * U * (np.abs(xh * c.gamma) + np.abs(c.beta))
        y = ref.activate(z, act)
        e_y = 1.1 * e_z + (2 * np.abs(z) + 8) * U * np.abs(y) + small.TINY
        small.inside(c.host(c.y), y, e_y + small.HALF["bf16"] * (np.abs(y) + e_y), "y")
        q, s = quantised(c)
        t, scale = ref.quantise_rows(y.reshape(-1, c.C))
        e_y = e_y.reshape(-1, c.C)
        e_top, a = e_y.max(axis=1), scale * 127.0
        small.inside(s.cpu().numpy(), scale, e_top / 127.0 + 4 * U * scale, "scale")
        tol = 0.5 + (127.0 / a)[:, None] * e_y + np.abs(t) * (e_top / a + 4 * U)[:, None] + 127 * 4 * U
        small.inside(q.view.cpu().numpy(), t, tol, "q")


@pytest.mark.parametrize("size", [(2, 64, 14, 14, 4), (1, 96, 20, 21, 3), (2, 40, 9, 11, 5), (1, 72, 31, 33, 9)], ids=str)
def test_constant_fp32_values(size):
    """The mean of equal values is that value, whatever its digits."""
    rng = np.random.default_rng(size[1])
    for value in np.exp(rng.uniform(0, 9, 8)).astype(np.float32):
        say(size, "f32", float(value))
        c = case(size, 0, "f32", lambda x: x.fill_(float(value)))
        c.forward()
        assert (c.mean.cpu() == float(value)).all()
        want = np.broadcast_to(c.beta.astype(np.float64), (c.N, c.P, c.C))
        np.testing.assert_array_equal(c.host(c.y), want)
