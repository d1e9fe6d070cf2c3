"""Rows of the layer norm that leave fp32's range: their statistics, values and scales are NaN, and no other row changes.

Bounds of the rows that stay inside it are test_gpu_layer_norm.py's.
"""

import numpy as np
import pytest
import torch

from block_helpers import close, draw, host, rounded, vec
from dora_weight_norm_amd import binding as bnd
from oracle import int8_oracle as Q
from test_gpu_layer_norm import EPS, bounds

pytestmark = pytest.mark.gpu
# a wave a row of one chunk and of two, 256, 512 and 1024 threads, and rows that are read again
SHAPES = [(600, 200), (600, 640), (9, 640), (520, 8192), (9, 8192), (9, 16000), (9, 20003)]


def out_of_range(x):
    """Rows 1 to 6: NaN, infinities, values whose sum or whose squares pass 2^128."""
    x[1, 3] = float("nan")
    x[2, 5], x[3, 7] = float("inf"), float("-inf")
    x[4] = 2.0 ** 127                     # the sum
    x[5] *= 2.0 ** 70                     # the squares
    x[6, 11] = 2.0 ** 100                 # the square of one
    return [1, 2, 3, 4, 5, 6]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_rows_past_the_range_are_nan(T, d, dtype):
    rng = np.random.default_rng(44)
    x, w, b = draw(rng, (T, d), dtype), vec(rng, d), vec(rng, d)
    clean = bnd.dora_layer_norm(x, w, b, EPS)
    clean8 = bnd.dora_layer_norm_quant(x, w, b, EPS)
    rows = out_of_range(x)
    keep = [t for t in range(T) if t not in rows]
    y, _, mean, rstd = bnd.dora_layer_norm(x, w, b, EPS)
    for v in (y, mean, rstd):
        assert torch.isnan(v[rows]).all()
    for got, want in zip((y, mean, rstd), (clean[0], clean[2], clean[3])):
        assert torch.equal(got[keep], want[keep])
    for q_dtype in (torch.int8, torch.float8_e4m3fn):
        q, scale, _, m, r = bnd.dora_layer_norm_quant(x, w, b, EPS, q_dtype=q_dtype)
        for v in (scale, m, r):
            assert torch.isnan(v[rows]).all()
        assert not q[rows].any() if q_dtype is torch.int8 else torch.isnan(q[rows].float()).all()
        if q_dtype is torch.int8:
            assert torch.equal(q[keep], clean8[0][keep]) and torch.equal(scale[keep], clean8[1][keep])


@pytest.mark.parametrize("T,d", SHAPES)
def test_large_rows_inside_the_range(T, d):
    """2^50 times normal values: d 2^100 is far from 2^128."""
    rng = np.random.default_rng(45)
    x, w, b = draw(rng, (T, d), "bf16", 2.0 ** 50), vec(rng, d), vec(rng, d)
    n, h, mean, rstd = Q.layer_norm(host(x), None, host(w), host(b), EPS)
    y, _, m, r = bnd.dora_layer_norm(x, w, b, EPS)
    em, er, en = bounds(n, h, mean, rstd, host(w), host(b))
    close(m, mean, em, "mean")
    close(r, rstd, er, "rstd")
    close(y, n, rounded("bf16", n, en), "y")
