"""The residual RMS norm and its backward on the GPU against the fp64 reference.

Tolerances. The fp32 sum of d squares in any order is off by at most
d 2^-24 relative, so rstd by half of that and the root's and division's few
roundings; n adds three roundings. Each output adds half a step of its type.
"""

import numpy as np
import pytest
import torch

from block_helpers import EPS32, TORCH_DT, close, draw, host, rounded, vec
from dora_weight_norm_amd import binding as bnd
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu
EPS = 1e-6
# (rows, elements): one wave, four rows a workgroup, every register shape, odd rows, the re-reading kernel
SHAPES = [(1, 1), (1, 7), (3, 8), (5, 513), (2, 511), (64, 256), (600, 1000), (513, 2048), (700, 2049), (520, 3583),
          (1, 4096), (7, 8192), (516, 8200), (1, 16384), (3, 16385), (2, 40003), (530, 16000), (0, 64),
          # more than 16 MiB of 16-bit rows: past the caches, several rows a workgroup
          (9000, 1000), (2200, 4100), (1040, 8200),
          # and in whole 128-byte lines
          (9000, 1024), (2100, 4096), (1030, 8192)]


def rel_n(d):
    return (0.5 * d + 8) * EPS32


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,d", SHAPES)
def test_norm(T, d, dtype):
    rng = np.random.default_rng(T * 100003 + d)
    x, res, w = draw(rng, (T, d), dtype, 0.5), draw(rng, (T, d), dtype), vec(rng, d)
    n, h, rstd = B.rms_norm(host(x), host(res), host(w), EPS)
    y, h2, r2 = bnd.dora_rms_norm(x, w, EPS, residual=res)
    e = np.abs(n) * rel_n(d)
    close(r2, rstd, rstd * rel_n(d), "rstd")
    close(h2, h, rounded(dtype, h, np.abs(h) * EPS32), "h")
    # (n's own fp32 sum x + residual is off by 2^-24 of h)
    close(y, n, rounded(dtype, n, e), "y")
    q, scale, h3, r3 = bnd.dora_rms_norm_quant(x, w, EPS, residual=res)
    assert torch.equal(h3, h2) and torch.equal(r3, r2)
    if T == 0:
        return
    top = np.abs(n).max(1)
    close(scale, top / 448, top / 448 * (rel_n(d) + 2 * EPS32), "scale")
    v = n / host(scale)[:, None]
    # half an e4m3 step (2^-4 of the value, 2^-10 below 2^-6) and n's fp32 error
    close(q, v, np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) + np.abs(v) * (rel_n(d) + 4 * EPS32), "q")


@pytest.mark.parametrize("T,d", [(4, 700), (600, 256), (2, 20000)])
def test_norm_without_residual_or_weight(T, d):
    rng = np.random.default_rng(5)
    x = draw(rng, (T, d), "bf16")
    n, _, rstd = B.rms_norm(host(x), None, None, EPS)
    y, h, r = bnd.dora_rms_norm(x, None, EPS)
    assert h is x
    close(r, rstd, rstd * rel_n(d), "rstd")
    close(y, n, rounded("bf16", n, np.abs(n) * rel_n(d)), "y")
    y2, _, none = bnd.dora_rms_norm(x, None, EPS, want_rstd=False)
    assert none is None and torch.equal(y2, y)


@pytest.mark.parametrize("T,d", [(3, 100), (520, 512), (2, 8192), (2, 17000)])
def test_norm_in_place_and_deterministic(T, d):
    rng = np.random.default_rng(6)
    x, res, w = draw(rng, (T, d), "bf16"), draw(rng, (T, d), "bf16"), vec(rng, d)
    want = bnd.dora_rms_norm_quant(x, w, EPS, residual=res)
    for into in ("x", "residual"):
        a, b = x.clone(), res.clone()
        got = bnd.dora_rms_norm_quant(a, w, EPS, residual=b, h=a if into == "x" else b)
        for g, r in zip(got, want):
            assert torch.equal(g.view(torch.uint8), r.view(torch.uint8)), into


@pytest.mark.parametrize("T,d", [(6, 640), (600, 640), (6, 18000)])
def test_norm_special_rows(T, d):
    rng = np.random.default_rng(7)
    x = draw(rng, (T, d), "bf16")
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] = 0
    x[3, 1] = 1e-38
    q, scale, _, rstd = bnd.dora_rms_norm_quant(x, None, EPS)
    y, _, _ = bnd.dora_rms_norm(x, None, EPS)
    s, f = host(scale), host(q)
    assert s[0] == 1 and (f[0] == 0).all() and (host(y)[0] == 0).all()
    assert np.isnan(s[1]) and np.isnan(f[1]).all() and np.isnan(host(y)[1]).all()
    assert host(rstd)[2] == 0 and np.isnan(host(y)[2, 5]) and (np.delete(host(y)[2], 5) == 0).all() and np.isnan(s[2])
    assert s[3] == 2.0 ** -100 and np.isfinite(f[3]).all()
    assert np.isfinite(f[4:]).all() and np.isfinite(s[4:]).all()


def test_norm_unaligned_tensors():
    """Views that start one element into a buffer: the same values as aligned ones."""
    rng = np.random.default_rng(8)
    T, d = 5, 264
    x, res, w = draw(rng, (T, d), "f16"), draw(rng, (T, d), "f16"), vec(rng, d)
    want = bnd.dora_rms_norm(x, w, EPS, residual=res)

    def off(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        b.copy_(t)
        return b

    got = bnd.dora_rms_norm(off(x), off(w), EPS, residual=off(res), y=off(x), h=off(x))
    for g, r in zip(got, want):
        assert torch.equal(g, r)


def bwd_tol(dy, h, rstd, w, dx, dh, dtype):
    d = dy.shape[1]
    a = np.abs(dy if w is None else dy * w)
    nh = np.abs(h) * rstd[:, None]
    err = rstd[:, None] * (6 * EPS32 * a + nh * ((d + 8) * EPS32 * np.mean(a * nh, 1, keepdims=True)))
    if dh is not None:
        err = err + EPS32 * np.abs(dx)
    return rounded(dtype, dx, err)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,d", [s for s in SHAPES if s[0] > 0] + [(2100, 300), (1100, 1500)])
def test_norm_backward(T, d, dtype):
    rng = np.random.default_rng(T * 7 + d)
    dy, h, dh, w = (draw(rng, (T, d), dtype), draw(rng, (T, d), dtype), draw(rng, (T, d), dtype), vec(rng, d))
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    H = [host(v) for v in (dy, h, rstd, w, dh)]
    dx, dw = B.rms_norm_backward(*H)
    gx, gw = bnd.dora_rms_norm_backward(dy, h, rstd, w, dh=dh)
    close(gx, dx, bwd_tol(H[0], H[1], H[2], H[3], dx, H[4], dtype), "dx")
    # T products of two roundings, added in any order
    close(gw, dw, (T + 4) * EPS32 * (np.abs(H[0]) * np.abs(H[1]) * H[2][:, None]).sum(0) + 1e-30, "dweight")
    only, none = bnd.dora_rms_norm_backward(dy, h, rstd, None, need_dweight=False)
    assert none is None
    dx1, _ = B.rms_norm_backward(H[0], H[1], H[2], None)
    close(only, dx1, bwd_tol(H[0], H[1], H[2], None, dx1, None, dtype), "dx without weight and dh")
    again = dy.clone()
    bnd.dora_rms_norm_backward(again, h, rstd, w, dh=dh, dx=again)
    assert torch.equal(again, gx)


def test_norm_backward_without_rows():
    z = torch.empty(0, 96, device="cuda")
    dx, dw = bnd.dora_rms_norm_backward(z, z, torch.empty(0, device="cuda"), None)
    assert dx.shape == (0, 96) and (dw == 0).all()


def test_norm_gradient_against_differences():
    """fp32 gradients of sum(n dy) + sum(h dh) against central differences of the fp64 reference."""
    rng = np.random.default_rng(9)
    T, d = 6, 70
    x, res, dy, dh, w = *(draw(rng, (T, d), "f32") for _ in range(4)), vec(rng, d)
    _, h, rstd = bnd.dora_rms_norm(x, w, EPS, residual=res)
    gx, gw = bnd.dora_rms_norm_backward(dy, h, rstd, w, dh=dh)

    def loss(xv, wv):
        n, hh, _ = B.rms_norm(xv, host(res), wv, EPS)
        return (n * host(dy)).sum() + (hh * host(dh)).sum()

    for _ in range(4):
        v, u, e = rng.standard_normal((T, d)), rng.standard_normal(d), 1e-5
        num = (loss(host(x) + e * v, host(w)) - loss(host(x) - e * v, host(w))) / (2 * e)
        assert abs((host(gx) * v).sum() - num) <= 1e-4 * np.linalg.norm(host(gx)) * np.linalg.norm(v)
        num = (loss(host(x), host(w) + e * u) - loss(host(x), host(w) - e * u)) / (2 * e)
        assert abs((host(gw) * u).sum() - num) <= 1e-4 * np.linalg.norm(host(gw)) * np.linalg.norm(u)


def test_norm_on_another_stream():
    rng = np.random.default_rng(10)
    x, res, w = draw(rng, (64, 1024), "bf16"), draw(rng, (64, 1024), "bf16"), vec(rng, 1024)
    want = bnd.dora_rms_norm(x, w, EPS, residual=res)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = bnd.dora_rms_norm(x, w, EPS, residual=res, stream=st)
    st.synchronize()
    for g, r in zip(got, want):
        assert torch.equal(g, r)


def test_norm_refuses_wrong_buffers():
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda")
    for bad in (dict(residual=x.float()), dict(residual=x[:3]), dict(residual=x, h=x.float()), dict(h=x),
                dict(y=x[:, ::2]), dict(rstd=w)):
        with pytest.raises((ValueError, TypeError)):
            bnd.dora_rms_norm(x, w, EPS, **bad)
    with pytest.raises(ValueError):
        bnd.dora_rms_norm(x, w[:32], EPS)
    with pytest.raises(ValueError):
        bnd.dora_rms_norm(x.t(), w[:4], EPS)
    with pytest.raises(TypeError):
        bnd.dora_rms_norm(x.double(), w, EPS)
    with pytest.raises(bnd.DoraError):
        bnd.dora_rms_norm(x, w, 0.0)
    with pytest.raises(bnd.DoraError):
        bnd.dora_rms_norm(x, w, EPS, y=x)


@pytest.mark.parametrize("T,d", [(3, 700), (600, 640), (64, 8192), (2, 20000)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_8_bit_rows_are_the_nearest_to_the_quotient(T, d, dtype):
    """q is the fp32 quotient n / scale, rounded once: bit by bit, on values beside the borders of the 8-bit steps."""
    rng = np.random.default_rng(T + d)
    # borders between neighbouring e4m3 values (17, 19, .. 31 in units of a half step) at a few exponents, each off
    # by an fp32 step or so
    edge = (17 + 2 * rng.integers(0, 8, (T, d))) * 2.0 ** rng.integers(-3, 4, (T, d)) * rng.choice([-1, 1], (T, d))
    edge[:, 0] = 448
    row = np.exp(rng.uniform(-2, 2, (T, 1))) / 100
    w = torch.from_numpy((1 + 0.3 * rng.random(d)).astype(np.float32)).cuda()
    x = torch.from_numpy((edge * row / (1 if dtype != "f32" else host(w)[None])).astype(np.float32)).cuda()
    x = x.to(TORCH_DT[dtype])
    if dtype != "f32":
        w = None
    q, scale, h, rstd = bnd.dora_rms_norm_quant(x, w, 1e-6)
    f = np.float32
    n = x.float().cpu().numpy() * rstd.cpu().numpy()[:, None]
    if w is not None:
        n = n * w.cpu().numpy()[None]
    assert n.dtype == f
    assert np.array_equal(scale.cpu().numpy(), np.abs(n).max(1) / f(448))
    want = torch.from_numpy(n / scale.cpu().numpy()[:, None]).to(torch.float8_e4m3fn)
    off = (q.cpu().float() != want.float())
    assert not off.any(), f"{off.sum()} of {off.numel()} values"


def test_8_bit_rows_of_infinite_scale():
    """n past fp32's range: its scale is infinite, the finite values are 0 and the infinite ones NaN."""
    x = torch.ones(2, 600, device="cuda")
    x[:, 7] = -2
    w = torch.full((600,), 3.0e38, device="cuda")
    w[100:] = 1
    q, scale, _, _ = bnd.dora_rms_norm_quant(x, w, EPS)
    v = host(q)
    assert np.isinf(host(scale)).all()
    assert np.isnan(v[:, 7]).all() and (np.delete(v, 7, 1) == 0).all()


@pytest.mark.parametrize("down", [60, 88, 100])
def test_8_bit_rows_of_tiny_values(down):
    """As above with n near 2^-down, past which the scale stays at 2^-100."""
    rng = np.random.default_rng(down)
    T, d, f = 40, 4000, np.float32
    x = draw(rng, (T, d), "f32")
    w = torch.from_numpy((rng.random(d) + 0.5).astype(f) * f(2.0 ** -down)).cuda()
    q, scale, _, rstd = bnd.dora_rms_norm_quant(x, w, 1e-6)
    n = x.cpu().numpy() * rstd.cpu().numpy()[:, None] * w.cpu().numpy()[None]
    assert np.array_equal(scale.cpu().numpy(), np.maximum(np.abs(n).max(1) / f(448), f(2.0 ** -100)))
    want = torch.from_numpy(n / scale.cpu().numpy()[:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(q.cpu().float(), want.float())


def test_offsets_past_32_bits():
    T, d, n = 270001, 8200, 40
    rng = np.random.default_rng(12)
    x, w = torch.zeros(T, d, device="cuda", dtype=torch.bfloat16), vec(rng, d)
    x[-n:] = draw(rng, (n, d), "bf16")
    want = bnd.dora_rms_norm_quant(x[-n:].clone(), w, EPS)
    q, scale, _, rstd = bnd.dora_rms_norm_quant(x, w, EPS)
    y, _, _ = bnd.dora_rms_norm(x, w, EPS)
    ref, _, _ = B.rms_norm(host(x[-n:]), None, host(w), EPS)
    close(y[-n:], ref, rounded("bf16", ref, np.abs(ref) * rel_n(d)), "y")
    close(scale[-n:], host(want[1]), host(want[1]) * 2 * rel_n(d), "scale")
    v = ref / host(scale[-n:])[:, None]
    close(q[-n:], v, np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) + np.abs(v) * (rel_n(d) + 4 * EPS32), "q")
    dx, dw = bnd.dora_rms_norm_backward(x, x, rstd, w, dx=y)
    rdx, rdw = B.rms_norm_backward(host(x[-n:]), host(x[-n:]), host(rstd[-n:]), host(w))
    close(dx[-n:], rdx, bwd_tol(host(x[-n:]), host(x[-n:]), host(rstd[-n:]), host(w), rdx, None, "bf16"), "dx")
    a = np.abs(host(x[-n:]))
    close(dw, rdw, (n + 4) * EPS32 * (a * a * host(rstd[-n:])[:, None]).sum(0) + 1e-30, "dweight")
    assert not dx[:-n].any()
