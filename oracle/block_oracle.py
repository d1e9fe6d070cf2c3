"""fp64 reference of the residual RMS norm and the matrix product with its
epilogue, and of their gradients (numpy, from the definitions; nothing shared
with the library)."""

from __future__ import annotations

import math

import numpy as np

try:
    from scipy.special import erf as _erf
except ImportError:   # pragma: no cover
    _erf = np.vectorize(math.erf)

E4M3_MAX = 448.0


def rms_norm(x, residual, weight, eps):
    """(n, h, rstd) in fp64; residual and weight may be None."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    n = h * rstd[:, None]
    if weight is not None:
        n = n * np.asarray(weight, np.float64)[None, :]
    return n, h, rstd


def rms_norm_backward(dy, h, rstd, weight, dh=None):
    """(dx, dweight) in fp64 from h and rstd."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    nh = h * np.asarray(rstd, np.float64)[:, None]
    a = dy if weight is None else dy * np.asarray(weight, np.float64)[None, :]
    dx = np.asarray(rstd, np.float64)[:, None] * (a - nh * np.mean(a * nh, axis=1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * nh).sum(0)


def _logistic(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def act(z, name):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * _logistic(z)
    assert name == "none"
    return z


def slope(z, name):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        th = np.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * k * (1.0 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = _logistic(z)
        return p + z * p * (1.0 - p)
    assert name == "none"
    return np.ones_like(z)


def product(x, w, row_scale=None, t=None, b=None, s=1.0):
    """u = row_scale (x w^T + s t b^T) in fp64."""
    u = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if t is not None:
        u = u + s * (np.asarray(t, np.float64) @ np.asarray(b, np.float64).T)
    if row_scale is not None:
        u = u * np.asarray(row_scale, np.float64)[:, None]
    return u


def preactivation(u, col_scale=None, bias=None):
    z = np.asarray(u, np.float64)
    if col_scale is not None:
        z = z * np.asarray(col_scale, np.float64)[None, :]
    if bias is not None:
        z = z + np.asarray(bias, np.float64)[None, :]
    return z


def matmul(x, w, row_scale=None, col_scale=None, t=None, b=None, s=1.0, bias=None, name="none", residual=None):
    """(y, u) in fp64."""
    u = product(x, w, row_scale, t, b, s)
    y = act(preactivation(u, col_scale, bias), name)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
    return y, u


def matmul_backward(dy, u, x, w, col_scale=None, bias=None, name="none"):
    """(dx, dw, dbias, dcol_scale, du) in fp64."""
    u = np.asarray(u, np.float64)
    dz = np.asarray(dy, np.float64) * slope(preactivation(u, col_scale, bias), name)
    du = dz if col_scale is None else dz * np.asarray(col_scale, np.float64)[None, :]
    return du @ np.asarray(w, np.float64), du.T @ np.asarray(x, np.float64), dz.sum(0), (dz * u).sum(0), du
