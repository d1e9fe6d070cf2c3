"""The fp64 reference of the layer norm and of int8 rows against autograd, differences and hand-made rows."""

import numpy as np
import torch

from oracle import int8_oracle as Q


def test_layer_norm_gradients_follow_autograd():
    rng = np.random.default_rng(1)
    T, d = 5, 37
    x, dy, dh = (rng.standard_normal((T, d)) for _ in range(3))
    w, b = 1 + 0.1 * rng.standard_normal(d), rng.standard_normal(d)
    tx, tw, tb = (torch.tensor(v, requires_grad=True) for v in (x, w, b))
    mu = tx.mean(1, keepdim=True)
    n = (tx - mu) / ((tx - mu).square().mean(1, keepdim=True) + 1e-5).sqrt() * tw + tb
    ((n * torch.tensor(dy)).sum() + (tx * torch.tensor(dh)).sum()).backward()
    ref, h, mean, rstd = Q.layer_norm(x, None, w, b, 1e-5)
    assert np.allclose(ref, n.detach().numpy(), atol=1e-12)
    dx, dw, db = Q.layer_norm_backward(dy, h, mean, rstd, w, dh)
    for g, t in ((dx, tx), (dw, tw), (db, tb)):
        assert np.allclose(g, t.grad.numpy(), atol=1e-11)


def test_a_constant_row_is_its_bias():
    n, _, mean, rstd = Q.layer_norm(np.full((1, 8), 3.0), None, np.ones(8), np.arange(8.0), 1e-4)
    assert mean[0] == 3 and np.isclose(rstd[0], 100) and np.array_equal(n[0], np.arange(8.0))


def test_int8_rows_by_hand():
    q, s = Q.quantize_rows([[127.0, 63.5, -0.5, 1.5, -127.0]])
    assert s[0] == 1 and np.array_equal(q[0], [127, 64, 0, 2, -127])      # ties to the even step
    q, s = Q.quantize_rows(np.zeros((2, 3)))
    assert (s == 1).all() and not q.any()
    x = np.concatenate([np.full((1, 32), 127.0), np.full((1, 8), 254.0)], axis=1)
    q, s = Q.quantize_rows(x, 32)
    assert s.shape == (1, 2) and np.array_equal(s[0], [1, 2]) and (q == 127).all()
    assert np.array_equal(Q.dequantize_rows(q, s, 32), x)


def test_int8_rows_are_within_half_a_step():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((7, 300)) * np.exp(rng.uniform(-20, 20, (7, 1)))
    for group in (0, 32, 64, 128, 256):
        q, s = Q.quantize_rows(x, group)
        assert np.abs(q).max() == 127
        step = np.abs(Q.dequantize_rows(np.ones_like(q), s, group))
        assert (np.abs(Q.dequantize_rows(q, s, group) - x) <= step * (0.5 + 127 * 2.0 ** -24)).all()
