"""Plain fp64 definitions of the operators beside the convolutions: group norm
with an activation (forward, backward), rows in 8 bits, integer products, RMS
norm, products with an epilogue and their gradients, dropout.

numpy only, written from the formulas in include/conv2d.h.  Activations are
[N, P, C] arrays (P = H*W pixels, channels last).
"""
from __future__ import annotations

import math

import numpy as np

ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU = 0, 1, 2, 3
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


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def normal_below(z):
    """The standard normal's distribution function."""
    return _erfc(-np.asarray(z, np.float64) / np.sqrt(2)) / 2


def activate(z, act):
    if act == ACT_RELU:
        return np.where(z < 0, 0.0, z)
    if act == ACT_SILU:
        return z * sigmoid(z)
    if act == ACT_GELU:
        return z * normal_below(z)
    return z


def activation_slope(z, act):
    if act == ACT_RELU:
        return (z > 0).astype(np.float64)
    if act == ACT_SILU:
        s = sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    if act == ACT_GELU:
        return normal_below(z) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
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


def rms_norm(x, residual, gamma, eps):
    """h, y, rstd of the rows of x + residual [M, C]; residual and gamma may be None."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    y = h * rstd[:, None]
    return h, y if gamma is None else y * np.asarray(gamma, np.float64), rstd


def rms_norm_bwd(dy, dh, h, gamma, rstd):
    """dx, dgamma for the given rstd [M]; dh and gamma may be None."""
    dy, r = np.asarray(dy, np.float64), np.asarray(rstd, np.float64)[:, None]
    xh = np.asarray(h, np.float64) * r
    t = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    dx = r * (t - xh * (t * xh).mean(axis=1, keepdims=True))
    return dx if dh is None else dx + np.asarray(dh, np.float64), (dy * xh).sum(axis=0)


def matmul(x, w, bias, residual, act):
    """y, z = act(z) + residual, x w^T + bias; bias and residual may be None."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    y = activate(z, act)
    return y if residual is None else y + np.asarray(residual, np.float64), z


def matmul_bwd(dy, z, x, w, act):
    """dx, dw, dbias, dz; z is not read without an activation."""
    dz = np.asarray(dy, np.float64)
    if act != ACT_NONE:
        dz = dz * activation_slope(np.asarray(z, np.float64), act)
    return dz @ np.asarray(w, np.float64), dz.T @ np.asarray(x, np.float64), dz.sum(axis=0), dz


def philox(counter, key, rounds=10):
    """Philox4x32: four words of a counter (integers or arrays of them) under a key of two."""
    c = [np.asarray(v, np.uint64) for v in counter]
    k = [int(v) for v in key]
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> half) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_keep(M, C, p, seed, offset, row0=0):
    """Which elements [M, C] of the rows from row0 on stay; p as the fp32 that the entry takes."""
    groups = -(-C // 4)
    words = philox([np.arange(groups)[None, :], (row0 + np.arange(M))[:, None], offset & 0xFFFFFFFF, offset >> 32],
                   [seed & 0xFFFFFFFF, seed >> 32])
    words = np.stack([np.broadcast_to(w, (M, groups)) for w in words], axis=2).reshape(M, -1)[:, :C]
    return words >= np.uint64(int(float(np.float32(p)) * 2.0 ** 32))


def dropout(x, residual, p, seed, offset):
    x = np.asarray(x, np.float64)
    y = np.where(dropout_keep(*x.shape, p, seed, offset), x / (1.0 - float(np.float32(p))), 0.0)
    return y if residual is None else y + np.asarray(residual, np.float64)
