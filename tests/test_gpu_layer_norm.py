"""The residual layer norm and its backward on the GPU against the fp64 reference.

Tolerances. The fp32 sum of d values in any order is off by at most d 2^-24 of
the mean of their sizes, which moves the mean; h itself, the sum of two, by
2^-24. The squares about that mean are off by (d + 4) 2^-24 relative, by the
square of the mean's error (their sum about the true mean is least), by what
moves a value in its own subtraction, and, where parts of a row are joined by
the squares of their means' distances, by twice the mean's error times such a
distance, whose root mean square is at most the spread. n then has three
roundings more. Each output adds half a step of its type.
"""

import numpy as np
import pytest
import torch

from block_helpers import EPS32, TORCH_DT, close, draw, host, rounded, vec
from dora_weight_norm_amd import binding as bnd
from oracle import int8_oracle as Q

pytestmark = pytest.mark.gpu
EPS = 1e-5
# (rows, elements): one wave, four rows a workgroup, every register shape, odd rows, the re-reading kernel
SHAPES = [(1, 1), (1, 7), (3, 8), (5, 513), (2, 511), (64, 256), (600, 1000), (513, 2048), (700, 2049), (520, 3583),
          (1, 4096), (7, 8192), (516, 8200), (1, 16384), (3, 16385), (2, 40003), (530, 16000), (0, 64),
          # more than 16 MiB of 16-bit rows: past the caches, several rows a workgroup
          (9000, 1000), (2200, 4100), (1040, 8200),
          # and in whole 128-byte lines
          (9000, 1024), (2100, 4096), (1030, 8192)]


def bounds(n, h, mean, rstd, w, b):
    """(error of the mean [T], of rstd [T], of n [T, d]) of fp32 arithmetic in any order."""
    d = h.shape[1]
    ah, v = np.abs(h), np.abs(h - mean[:, None])
    em = (d + 3) * EPS32 * ah.mean(1)
    move = EPS32 * (ah + v)                          # of one value in its sum and its subtraction
    var = (v * v).mean(1)
    evar = (d + 4) * EPS32 * (var + em * em) + em * em + 2 * (v * move).mean(1) + 2 * em * move.mean(1) + (move * move).mean(1)
    evar = evar + 2 * em * np.sqrt(var)
    # (the square root halves a small relative error; a large one, of a variance near 0, is taken whole)
    rel = evar * rstd * rstd
    erel = np.where(rel < 0.1, 0.6 * rel, 2 * rel) + 4 * EPS32
    W = 1.0 if w is None else np.abs(w)[None, :]
    body = v * rstd[:, None] * W
    en = W * (rstd * (1 + erel))[:, None] * (em[:, None] + move) + body * (erel[:, None] + 4 * EPS32) + EPS32 * np.abs(n)
    return em, rstd * erel, en


def check_8_bits(q, scale, n, en, q_dtype):
    top, at = np.abs(n).max(1), np.abs(n) + en
    most = 127 if q_dtype is torch.int8 else 448
    close(scale, top / most, at.max(1) * 2 * EPS32 / most + en.max(1) / most, "scale")
    s = host(scale)[:, None]
    v, ev = n / s, en / s + 4 * EPS32 * np.abs(n) / s
    if q_dtype is torch.int8:
        assert np.abs(host(q)).max() <= 127
        close(q, v, 0.5 + ev, "q")
    else:   # half an e4m3 step: 2^-4 of the value, 2^-10 below 2^-6
        close(q, v, np.maximum((np.abs(v) + ev) * 2.0 ** -4, 2.0 ** -10) + ev, "q")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_layer_norm(T, d, dtype):
    rng = np.random.default_rng(T * 100003 + d)
    x, res, w, b = draw(rng, (T, d), dtype, 0.5, 0.3), draw(rng, (T, d), dtype), vec(rng, d), vec(rng, d, 0.2, 0.0)
    n, h, mean, rstd = Q.layer_norm(host(x), host(res), host(w), host(b), EPS)
    y, h2, m2, r2 = bnd.dora_layer_norm(x, w, b, EPS, residual=res)
    if T == 0:
        assert y.shape == (0, d) and m2.shape == (0,)
        return
    em, er, en = bounds(n, h, mean, rstd, host(w), host(b))
    close(m2, mean, em, "mean")
    close(r2, rstd, er, "rstd")
    close(h2, h, rounded(dtype, h, np.abs(h) * EPS32), "h")
    close(y, n, rounded(dtype, n, en), "y")
    for q_dtype in (torch.int8, torch.float8_e4m3fn):
        both = torch.empty_like(x)
        q, scale, h3, m3, r3 = bnd.dora_layer_norm_quant(x, w, b, EPS, q_dtype=q_dtype, residual=res, y=both)
        assert torch.equal(h3, h2) and torch.equal(m3, m2) and torch.equal(r3, r2) and torch.equal(both, y)
        check_8_bits(q, scale, n, en, q_dtype)


@pytest.mark.parametrize("T,d", [(4, 700), (600, 256), (2, 20000)])
def test_layer_norm_without_residual_weight_or_bias(T, d):
    rng = np.random.default_rng(5)
    x = draw(rng, (T, d), "bf16")
    n, h, mean, rstd = Q.layer_norm(host(x), None, None, None, EPS)
    y, h2, m, r = bnd.dora_layer_norm(x, None, None, EPS)
    assert h2 is x
    close(y, n, rounded("bf16", n, bounds(n, h, mean, rstd, None, None)[2]), "y")
    y2, _, a, b = bnd.dora_layer_norm(x, None, None, EPS, want_stats=False)
    assert a is None and b is None and torch.equal(y2, y)
    w, b = vec(rng, d), vec(rng, d)
    for ww, bb in ((w, None), (None, b)):
        n, h, mean, rstd = Q.layer_norm(host(x), None, host(ww), host(bb), EPS)
        close(bnd.dora_layer_norm(x, ww, bb, EPS)[0], n,
              rounded("bf16", n, bounds(n, h, mean, rstd, host(ww), host(bb))[2]), "y")


@pytest.mark.parametrize("T,d", [(3, 100), (600, 1000), (4, 8192), (2, 17000)])
def test_a_mean_far_larger_than_the_spread(T, d):
    """Rows of 1000 +- 1: a sum of squares less the square of the sum would lose the variance's digits."""
    rng = np.random.default_rng(6)
    x, w, b = draw(rng, (T, d), "f32", 1.0, 1000.0), vec(rng, d), vec(rng, d)
    n, h, mean, rstd = Q.layer_norm(host(x), None, host(w), host(b), EPS)
    y, _, m, r = bnd.dora_layer_norm(x, w, b, EPS)
    em, er, en = bounds(n, h, mean, rstd, host(w), host(b))
    close(m, mean, em, "mean")
    close(r, rstd, er, "rstd")
    close(y, n, rounded("f32", n, en), "y")
    # (sums over a wave's lanes and a thread's few values are far better than d in a row)
    assert np.abs(host(r) / rstd - 1).max() < 1e-5


@pytest.mark.parametrize("T,d", [(3, 100), (520, 512), (2, 8192), (2, 17000)])
def test_layer_norm_in_place_and_deterministic(T, d):
    rng = np.random.default_rng(6)
    x, res, w, b = draw(rng, (T, d), "bf16"), draw(rng, (T, d), "bf16"), vec(rng, d), vec(rng, d)
    want = bnd.dora_layer_norm_quant(x, w, b, EPS, residual=res)
    for into in ("x", "residual"):
        u, v = x.clone(), res.clone()
        got = bnd.dora_layer_norm_quant(u, w, b, EPS, residual=v, h=u if into == "x" else v)
        for g, r in zip(got, want):
            assert torch.equal(g, r), into


@pytest.mark.parametrize("T,d", [(7, 640), (600, 640), (7, 18000)])
def test_layer_norm_special_rows(T, d):
    rng = np.random.default_rng(7)
    x = draw(rng, (T, d), "bf16")
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] = 1.5                        # no spread
    x[4] = 0
    x[4, 1] = 1e-38
    y, _, mean, rstd = bnd.dora_layer_norm(x, None, None, EPS)
    top = EPS ** -0.5
    assert (host(y)[[0, 3]] == 0).all() and np.allclose(host(rstd)[[0, 3]], top, rtol=1e-6) and host(mean)[3] == 1.5
    assert np.isnan(host(y)[1]).all() and np.isnan(host(y)[2]).all()
    assert np.isfinite(host(y)[5:]).all()
    q, scale, _, _, _ = bnd.dora_layer_norm_quant(x, None, None, EPS)
    s = host(scale)
    assert (s[[0, 3]] == 1).all() and np.isnan(s[[1, 2]]).all() and (host(q)[:4] == 0).all()
    assert s[4] == 2.0 ** -100 and np.isfinite(s[5:]).all()
    q, scale, _, _, _ = bnd.dora_layer_norm_quant(x, None, None, EPS, q_dtype=torch.float8_e4m3fn)
    assert np.isnan(host(q)[1]).all() and np.isnan(host(q)[2]).all() and np.isfinite(host(q)[5:]).all()


def off(t):
    """The same values one element into a buffer."""
    b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
    b.copy_(t)
    return b


@pytest.mark.parametrize("d", [264, 777])
def test_layer_norm_unaligned_tensors(d):
    rng = np.random.default_rng(8)
    T = 5
    x, res, w, b = draw(rng, (T, d), "f16"), draw(rng, (T, d), "f16"), vec(rng, d), vec(rng, d)
    want = bnd.dora_layer_norm(x, w, b, EPS, residual=res)
    got = bnd.dora_layer_norm(off(x), off(w), off(b), EPS, residual=off(res), y=off(x), h=off(x))
    for g, r in zip(got, want):
        assert torch.equal(g, r)
    wq = bnd.dora_layer_norm_quant(x, w, b, EPS, residual=res)
    gq = bnd.dora_layer_norm_quant(off(x), off(w), off(b), EPS, residual=off(res), q=off(wq[0]))
    assert torch.equal(gq[0], wq[0]) and torch.equal(gq[1], wq[1])


def bwd_tol(dy, h, mean, rstd, w, dx, dh, dtype):
    d = dy.shape[1]
    a = np.abs(dy if w is None else dy * w)
    nh = np.abs(h - mean[:, None]) * rstd[:, None]
    err = rstd[:, None] * (8 * EPS32 * a + (d + 6) * EPS32 * a.mean(1, keepdims=True)
                           + nh * ((d + 10) * EPS32 * np.mean(a * nh, 1, keepdims=True)))
    if dh is not None:
        err = err + EPS32 * np.abs(dx)
    return rounded(dtype, dx, err)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,d", [s for s in SHAPES if s[0] > 0] + [(2100, 300), (1100, 1500)])
def test_layer_norm_backward(T, d, dtype):
    rng = np.random.default_rng(T * 7 + d)
    dy, h, dh, w = (draw(rng, (T, d), dtype), draw(rng, (T, d), dtype, 1.0, 0.4), draw(rng, (T, d), dtype), vec(rng, d))
    mean = h.double().mean(1).float()
    rstd = ((h.double() - mean.double()[:, None]).square().mean(1) + EPS).rsqrt().float()
    H = [host(v) for v in (dy, h, mean, rstd, w, dh)]
    dx, dw, db = Q.layer_norm_backward(*H)
    gx, gw, gb = bnd.dora_layer_norm_backward(dy, h, mean, rstd, w, dh=dh)
    close(gx, dx, bwd_tol(H[0], H[1], H[2], H[3], H[4], dx, H[5], dtype), "dx")
    # T products of four roundings, added in any order
    close(gw, dw, (T + 6) * EPS32 * (np.abs(H[0]) * np.abs(H[1] - H[2][:, None]) * H[3][:, None]).sum(0) + 1e-30, "dweight")
    close(gb, db, (T + 1) * EPS32 * np.abs(H[0]).sum(0), "dbias")
    only, n1, n2 = bnd.dora_layer_norm_backward(dy, h, mean, rstd, None, need_dweight=False, need_dbias=False)
    assert n1 is None and n2 is None
    dx1, _, _ = Q.layer_norm_backward(H[0], H[1], H[2], H[3], None)
    close(only, dx1, bwd_tol(H[0], H[1], H[2], H[3], None, dx1, None, dtype), "dx without weight and dh")
    again = dy.clone()
    _, w2, b2 = bnd.dora_layer_norm_backward(again, h, mean, rstd, w, dh=dh, dx=again)
    assert torch.equal(again, gx) and torch.equal(w2, gw) and torch.equal(b2, gb)
    _, w3, none = bnd.dora_layer_norm_backward(dy, h, mean, rstd, w, dh=dh, need_dbias=False)
    assert none is None and torch.equal(w3, gw)
    _, none, b3 = bnd.dora_layer_norm_backward(dy, h, mean, rstd, w, dh=dh, need_dweight=False)
    assert none is None and torch.equal(b3, gb)


def test_layer_norm_backward_without_rows():
    z, e = torch.empty(0, 96, device="cuda"), torch.empty(0, device="cuda")
    stale = [torch.full((n,), float("nan"), device="cuda") for n in (96, 96, 192)]
    del stale
    dx, dw, db = bnd.dora_layer_norm_backward(z, z, e, e, None)
    assert dx.shape == (0, 96) and (dw == 0).all() and (db == 0).all()


def test_layer_norm_gradient_against_differences():
    """fp32 gradients of sum(n dy) + sum(h dh) against central differences of the fp64 reference."""
    rng = np.random.default_rng(9)
    T, d = 6, 70
    x, res, dy, dh, w, b = *(draw(rng, (T, d), "f32") for _ in range(4)), vec(rng, d), vec(rng, d)
    _, h, mean, rstd = bnd.dora_layer_norm(x, w, b, EPS, residual=res)
    gx, gw, gb = bnd.dora_layer_norm_backward(dy, h, mean, rstd, w, dh=dh)

    def loss(xv, wv, bv):
        n, hh, _, _ = Q.layer_norm(xv, host(res), wv, bv, EPS)
        return (n * host(dy)).sum() + (hh * host(dh)).sum()

    vals = [host(x), host(w), host(b)]
    for i, g in enumerate((gx, gw, gb)):
        for _ in range(4):
            v, e = rng.standard_normal(vals[i].shape), 1e-5
            up, down = ([vals[j] + s * e * v if j == i else vals[j] for j in range(3)] for s in (1, -1))
            num = (loss(*up) - loss(*down)) / (2 * e)
            assert abs((host(g) * v).sum() - num) <= 1e-4 * np.linalg.norm(host(g)) * np.linalg.norm(v), i


def test_layer_norm_on_another_stream():
    rng = np.random.default_rng(10)
    x, res, w, b = draw(rng, (64, 1024), "bf16"), draw(rng, (64, 1024), "bf16"), vec(rng, 1024), vec(rng, 1024)
    want = bnd.dora_layer_norm(x, w, b, EPS, residual=res)
    dwant = bnd.dora_layer_norm_backward(x, want[1], want[2], want[3], w)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = bnd.dora_layer_norm(x, w, b, EPS, residual=res, stream=st)
    dgot = bnd.dora_layer_norm_backward(x, got[1], got[2], got[3], w, stream=st)
    st.synchronize()
    for g, r in zip(got + dgot, want + dwant):
        assert torch.equal(g, r)


def test_layer_norm_refuses_wrong_buffers():
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda")
    for bad in (dict(residual=x.float()), dict(residual=x[:3]), dict(residual=x, h=x.float()), dict(h=x),
                dict(y=x[:, ::2]), dict(rstd=w), dict(mean=w)):
        with pytest.raises((ValueError, TypeError)):
            bnd.dora_layer_norm(x, w, w, EPS, **bad)
    for bad in (dict(q_dtype=torch.uint8), dict(q=x), dict(scale=w), dict(q=torch.zeros(4, 64, device="cuda").to(torch.float8_e4m3fn))):
        with pytest.raises((ValueError, TypeError)):
            bnd.dora_layer_norm_quant(x, w, w, EPS, **bad)
    with pytest.raises(ValueError):
        bnd.dora_layer_norm(x, w, w[:32], EPS)
    with pytest.raises(ValueError):
        bnd.dora_layer_norm(x.t(), w[:4], w[:4], EPS)
    with pytest.raises(TypeError):
        bnd.dora_layer_norm(x.double(), w, w, EPS)
    with pytest.raises(bnd.DoraError):
        bnd.dora_layer_norm(x, w, w, 0.0)
    with pytest.raises(bnd.DoraError):
        bnd.dora_layer_norm(x, w, w, EPS, y=x)
    s = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError):
        bnd.dora_layer_norm_backward(x, x, s, s, w, need_dbias=False, dbias=w)


def test_layer_norm_offsets_past_32_bits():
    T, d, n = 270001, 8200, 40
    rng = np.random.default_rng(12)
    x, w, b = torch.zeros(T, d, device="cuda", dtype=torch.bfloat16), vec(rng, d), vec(rng, d)
    x[-n:] = draw(rng, (n, d), "bf16")
    q, scale, _, mean, rstd = bnd.dora_layer_norm_quant(x, w, b, EPS)
    ref, h, m, r = Q.layer_norm(host(x[-n:]), None, host(w), host(b), EPS)
    en = bounds(ref, h, m, r, host(w), host(b))[2]
    check_8_bits(q[-n:], scale[-n:], ref, en, torch.int8)
    y, _, _, _ = bnd.dora_layer_norm(x, w, b, EPS)
    close(y[-n:], ref, rounded("bf16", ref, en), "y")
    y[:-n] = 0
    dx, dw, db = bnd.dora_layer_norm_backward(y, x, mean, rstd, w, dx=y)
    assert not dx[:-n].any()
    H = [host(ref_) for ref_ in (x[-n:], mean[-n:], rstd[-n:], w)]
    # (dx took y's place: its gradient is checked against the rounded y of the reference's tail)
    dy = torch.from_numpy(ref).cuda().to(torch.bfloat16)
    got, _, _ = bnd.dora_layer_norm_backward(dy, x[-n:].clone(), mean[-n:].clone(), rstd[-n:].clone(), w)
    rdx, _, _ = Q.layer_norm_backward(host(dy), H[0], H[1], H[2], H[3])
    close(got, rdx, bwd_tol(host(dy), H[0], H[1], H[2], H[3], rdx, None, "bf16"), "dx")
    # y rounds as ref's bf16 but where the fp32 error crosses a border: a step of 2^-7 of the value
    step = 2.0 ** -7 * np.abs(host(dy)).max()
    close(dx[-n:], host(got), 4 * H[2][:, None] * np.abs(H[3]).max() * step + 2.0 ** -7 * np.abs(host(got)), "dx far out")
