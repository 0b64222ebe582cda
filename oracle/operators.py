"""Plain fp64 definitions of the operators beside the convolutions: group norm
with an activation (forward, backward), rows in 8 bits, integer products.

numpy only, written from the formulas in include/conv2d.h.  Activations are
[N, P, C] arrays (P = H*W pixels, channels last).
"""
from __future__ import annotations

import numpy as np

ACT_NONE, ACT_RELU, ACT_SILU = 0, 1, 2
ROW_FLOOR = 2.0 ** -100


def _groups(a, G):
    N, P, C = a.shape
    return a.reshape(N, P, G, C // G)


def group_stats(x, G, eps):
    """mean, rstd [N, G] of x [N, P, C]."""
    v = _groups(np.asarray(x, np.float64), G)
    mean = v.mean(axis=(1, 3))
    var = ((v - mean[:, None, :, None]) ** 2).mean(axis=(1, 3))
    return mean, 1.0 / np.sqrt(var + eps)


def normalise(x, mean, rstd):
    """xh = (x - mean) * rstd, per group."""
    x = np.asarray(x, np.float64)
    G = mean.shape[1]
    v = _groups(x, G)
    return ((v - np.asarray(mean, np.float64)[:, None, :, None]) *
            np.asarray(rstd, np.float64)[:, None, :, None]).reshape(x.shape)


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def activate(z, act):
    if act == ACT_RELU:
        return np.where(z < 0, 0.0, z)
    if act == ACT_SILU:
        return z * sigmoid(z)
    return z


def activation_slope(z, act):
    if act == ACT_RELU:
        return (z > 0).astype(np.float64)
    if act == ACT_SILU:
        s = sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


def group_norm(x, gamma, beta, G, eps, act):
    """y, mean, rstd."""
    mean, rstd = group_stats(x, G, eps)
    z = normalise(x, mean, rstd) * np.asarray(gamma, np.float64) + np.asarray(beta, np.float64)
    return activate(z, act), mean, rstd


def group_norm_bwd(dy, x, gamma, beta, mean, rstd, act):
    """dx, dgamma, dbeta for the given mean and rstd [N, G]."""
    N, P, C = x.shape
    G = mean.shape[1]
    gamma = np.asarray(gamma, np.float64)
    xh = normalise(x, mean, rstd)
    z = xh * gamma + np.asarray(beta, np.float64)
    dz = np.asarray(dy, np.float64) * activation_slope(z, act)
    t = gamma * dz
    s1 = _groups(t, G).mean(axis=(1, 3))
    s2 = _groups(t * xh, G).mean(axis=(1, 3))
    per = lambda s: np.repeat(s, C // G, axis=1)[:, None, :]  # noqa: E731
    dx = per(np.asarray(rstd, np.float64)) * (t - per(s1) - xh * per(s2))
    return dx, (dz * xh).sum(axis=(0, 1)), dz.sum(axis=(0, 1))


def quantise_rows(v):
    """(the unrounded 127 v / a, the scale a / 127) of the rows of v [M, K]."""
    v = np.asarray(v, np.float64)
    a = np.maximum(np.abs(v).max(axis=1), ROW_FLOOR)
    return v * 127.0 / a[:, None], a / 127.0


def int8_matmul(q, q_scale, w, w_scale, bias=None, relu=False):
    """y [M, N], and the sum of the magnitudes of its two terms."""
    acc = np.asarray(q, np.int64) @ np.asarray(w, np.int64).T
    v = acc * (np.asarray(q_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64))
    size = np.abs(v)
    if bias is not None:
        b = np.asarray(bias, np.float64)
        v = v + b
        size = size + np.abs(b)
    return (np.where(v < 0, 0.0, v) if relu else v), size
