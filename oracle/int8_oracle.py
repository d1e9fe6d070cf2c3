"""fp64 reference of the layer norm and its gradients, and of rows held in
8-bit integers (numpy, from the definitions; nothing shared with the
library). The products are block_oracle's, on the values the rows stand for."""

from __future__ import annotations

import numpy as np

INT8_MAX = 127.0


def layer_norm(x, residual, weight, bias, eps):
    """(n, h, mean, rstd) in fp64; residual, weight and bias may be None."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    mean = h.mean(axis=1)
    v = h - mean[:, None]
    rstd = 1.0 / np.sqrt(np.mean(v * v, axis=1) + eps)
    n = v * rstd[:, None]
    if weight is not None:
        n = n * np.asarray(weight, np.float64)[None, :]
    if bias is not None:
        n = n + np.asarray(bias, np.float64)[None, :]
    return n, h, mean, rstd


def layer_norm_backward(dy, h, mean, rstd, weight, dh=None):
    """(dx, dweight, dbias) in fp64 from h, mean and rstd."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    rstd = np.asarray(rstd, np.float64)[:, None]
    nh = (h - np.asarray(mean, np.float64)[:, None]) * rstd
    a = dy if weight is None else dy * np.asarray(weight, np.float64)[None, :]
    dx = rstd * (a - a.mean(axis=1, keepdims=True) - nh * np.mean(a * nh, axis=1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * nh).sum(0), dy.sum(0)


def _columns(scale, d, group):
    """A scale [T] or [T, groups] at each of the d columns."""
    scale = np.asarray(scale, np.float64).reshape(len(scale), -1)
    return np.repeat(scale, group or d, axis=1)[:, :d]


def quantize_rows(x, group=0):
    """(q, scale): scale fp32 as it is held, q the whole numbers nearest to x / scale, ties to the even one."""
    x = np.asarray(x, np.float64)
    T, d = x.shape
    g = group or d
    n = -(-d // g)
    padded = np.concatenate([np.abs(x), np.zeros((T, n * g - d))], axis=1).reshape(T, n, g)
    top = padded.max(axis=2).astype(np.float32)
    scale = np.where(top == 0, np.float32(1), np.maximum(top / np.float32(INT8_MAX), np.float32(2.0 ** -100)))
    q = np.rint(x / _columns(scale, d, group))
    return q, (scale if group else scale.reshape(T))


def dequantize_rows(q, scale, group=0):
    q = np.asarray(q, np.float64)
    return q * _columns(scale, q.shape[1], group)
