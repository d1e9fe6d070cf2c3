"""The fp64 reference of the norm and product: hand values, and gradients against differences (CPU)."""

import numpy as np
import pytest

from oracle import block_oracle as B

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def test_rms_norm_by_hand():
    n, h, rstd = B.rms_norm([[3.0, 4.0]], [[0.0, 0.0]], [2.0, 1.0], 0.0)
    assert np.allclose(rstd, 1 / np.sqrt(12.5)) and np.allclose(n, [[6 / np.sqrt(12.5), 4 / np.sqrt(12.5)]])
    assert np.array_equal(h, [[3.0, 4.0]])


def test_activations_by_hand():
    assert B.act(1.0, "gelu") == pytest.approx(0.8413447460685429)
    assert B.act(1.0, "silu") == pytest.approx(0.7310585786300049)
    assert B.act(1.0, "gelu_tanh") == pytest.approx(0.8411919906082768)
    assert B.act(-2.0, "relu") == 0.0 and B.act(-2.0, "none") == -2.0


@pytest.mark.parametrize("name", ACTS)
def test_slopes_against_differences(name):
    z = np.linspace(-4, 4, 33) + 0.013
    e = 1e-6
    assert np.allclose(B.slope(z, name), (B.act(z + e, name) - B.act(z - e, name)) / (2 * e), atol=1e-8)


def _directional(f, v, d, e=1e-6):
    return (f(v + e * d) - f(v - e * d)) / (2 * e)


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, res, dy, dh = (rng.standard_normal((5, 7)) for _ in range(4))
    w = 1 + 0.1 * rng.standard_normal(7)

    def loss(x_, w_):
        n, h, _ = B.rms_norm(x_, res, w_, 1e-6)
        return (n * dy).sum() + (h * dh).sum()

    _, h, rstd = B.rms_norm(x, res, w, 1e-6)
    dx, dw = B.rms_norm_backward(dy, h, rstd, w, dh)
    for _ in range(4):
        d, e = rng.standard_normal(x.shape), rng.standard_normal(7)
        assert (dx * d).sum() == pytest.approx(_directional(lambda v: loss(v, w), x, d), rel=1e-6)
        assert (dw * e).sum() == pytest.approx(_directional(lambda v: loss(x, v), w, e), rel=1e-6)


@pytest.mark.parametrize("name", ACTS)
def test_product_gradients_against_differences(name):
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((6, 5)), rng.standard_normal((4, 5))
    c, bias, dy = 1 + 0.1 * rng.standard_normal(4), rng.standard_normal(4), rng.standard_normal((6, 4))

    def loss(x_=x, w_=w, c_=c, b_=bias):
        return (B.matmul(x_, w_, col_scale=c_, bias=b_, name=name)[0] * dy).sum()

    u = B.product(x, w)
    dx, dw, db, dc, _ = B.matmul_backward(dy, u, x, w, c, bias, name)
    for key, v, g in (("x_", x, dx), ("w_", w, dw), ("c_", c, dc), ("b_", bias, db)):
        d = rng.standard_normal(v.shape)
        assert (g * d).sum() == pytest.approx(_directional(lambda q: loss(**{key: q}), v, d), rel=1e-5, abs=1e-7)
