"""The feed-forward block: the norm and the products together, against the fp64 reference and against differences.

Tolerances. In fp32 every intermediate is off by a few K 2^-24 of its terms:
1e-4 of a result's norm covers five chained steps of these sizes with room.
In bf16 each of the up to eight roundings on the way is at most 2^-8 of a
value, 2^-8 of a tensor's norm: 8 * 2^-8; an 8-bit operand's rounding is 2^-4
of a value, two of them on the way to the up projection.
"""

import numpy as np
import pytest
import torch

from block_helpers import draw, host, vec
from dora_weight_norm_amd import binding as bnd
from dora_weight_norm_amd import block
from dora_weight_norm_amd.layer import dora_linear
from oracle import block_oracle as B
from oracle import dora_oracle as O

pytestmark = pytest.mark.gpu


def make(dtype, d, f, r, seed=0):
    rng = np.random.default_rng(seed)

    def layer(o, i):
        W, A, Bm = draw(rng, (o, i), dtype, i ** -0.5), draw(rng, (r, i), dtype, i ** -0.5), draw(rng, (o, r), dtype, 0.1)
        wn = O.dense_row_norm(host(W), host(A), host(Bm), 0.5)
        m = torch.from_numpy((wn * (1 + 0.05 * rng.standard_normal(o))).astype(np.float32)).cuda()
        return block.AdaptedLayer(W, A, Bm, m, 0.5, vec(rng, o, 0.1, 0.0))

    return block.FeedForward(vec(rng, d), layer(f, d), layer(d, f)), rng


def layer64(x, p, name="none", residual=None, **over):
    v = {k: over.get(k, host(getattr(p, k))) for k in ("W", "A", "B", "m", "bias")}
    # (the row norm is detached: of the layer as it is, not of the varied one)
    g = v["m"] / O.dense_row_norm(host(p.W), host(p.A), host(p.B), p.s)
    y, _ = B.matmul(x, v["W"], col_scale=g, t=x @ v["A"].T, b=v["B"], s=p.s, bias=v["bias"], name=name,
                    residual=residual)
    return y


def block64(x, res, p, nw=None, up=None, down=None):
    n, h, _ = B.rms_norm(x, res, host(p.norm_weight) if nw is None else nw, p.eps)
    a = layer64(n, p.up, p.act, **(up or {}))
    return layer64(a, p.down, residual=h, **(down or {}))


def rel(got, ref):
    return np.linalg.norm(host(got) - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("dtype,T,d,f,r", [("f32", 40, 64, 96, 8), ("bf16", 300, 264, 520, 24), ("f16", 1, 256, 384, 16),
                                           ("bf16", 7, 1000, 777, 5)])
def test_forward(dtype, T, d, f, r):
    p, rng = make(dtype, d, f, r)
    x, res = draw(rng, (T, d), dtype), draw(rng, (T, d), dtype)
    out, _ = block.forward(x, res, p)
    assert rel(out, block64(host(x), host(res), p)) <= (1e-4 if dtype == "f32" else 8 * 2.0 ** -8)


def test_gradients_against_differences():
    p, rng = make("f32", 48, 72, 8)
    x, res, dout = (draw(rng, (20, 48), "f32") for _ in range(3))
    _, saved = block.forward(x, res, p)
    g = block.backward(dout, saved, p)

    def loss(dx=0, dn=0, up=None, down=None):
        return (block64(host(x) + dx, host(res), p, host(p.norm_weight) + dn, up, down) * host(dout)).sum()

    def check(grad, f, what):
        d, e = rng.standard_normal(grad.shape), 1e-5
        num = (f(e * d) - f(-e * d)) / (2 * e)
        assert abs((host(grad) * d).sum() - num) <= 1e-4 * np.linalg.norm(host(grad)) * np.linalg.norm(d), what

    check(g["x"], lambda v: loss(dx=v), "x")
    check(g["norm_weight"], lambda v: loss(dn=v), "norm_weight")
    for side in ("up", "down"):
        layer = getattr(p, side)
        for k in ("A", "B", "m", "bias"):
            check(g[side][k], lambda v: loss(**{side: {k: host(getattr(layer, k)) + v}}), f"{side} {k}")


def test_bf16_gradients_follow_fp32():
    p, rng = make("bf16", 256, 512, 16)
    x, res, dout = (draw(rng, (128, 256), "bf16") for _ in range(3))
    _, s16 = block.forward(x, res, p)
    g16 = block.backward(dout, s16, p)
    wide = lambda q: block.AdaptedLayer(q.W.float(), q.A.float(), q.B.float(), q.m, q.s, q.bias)   # noqa: E731
    p32 = block.FeedForward(p.norm_weight, wide(p.up), wide(p.down))
    _, s32 = block.forward(x.float(), res.float(), p32)
    g32 = block.backward(dout.float(), s32, p32)
    for a, b in ((g16["x"], g32["x"]), (g16["norm_weight"], g32["norm_weight"]), (g16["up"]["A"], g32["up"]["A"]),
                 (g16["up"]["m"], g32["up"]["m"]), (g16["down"]["B"], g32["down"]["B"])):
        assert rel(a, host(b)) <= 16 * 2.0 ** -8      # (as many roundings back as forth)


@pytest.mark.parametrize("T", [1, 16, 200])
def test_8_bit_serving(T):
    p, rng = make("bf16", 512, 1024, 16)
    x, res = draw(rng, (T, 512), "bf16"), draw(rng, (T, 512), "bf16")
    _, g_down = p.down.magnitude()
    out = block.forward_8bit(x, res, p, block.freeze_8bit(p.up), g_down)
    assert rel(out, block64(host(x), host(res), p)) <= 2 * 2.0 ** -4 + 8 * 2.0 ** -8


def test_fused_layer_agrees_with_dora_linear():
    p, rng = make("bf16", 512, 768, 32)
    x = draw(rng, (300, 512), "bf16")
    q = block.AdaptedLayer(p.up.W, p.up.A, p.up.B, p.up.m, p.up.s)
    y, _, _ = block.adapted_linear(x, q, q.magnitude()[1])
    ref = dora_linear(x, q.W, q.A, q.B, q.m, q.s)
    assert rel(y, host(ref)) <= 3 * 2.0 ** -8         # (t, base, lora and y are rounded in the one, t and y in the other)


def test_block_on_a_stream_of_its_own():
    p, rng = make("bf16", 256, 512, 16)
    x, res, dout = (draw(rng, (64, 256), "bf16") for _ in range(3))
    want, saved = block.forward(x, res, p)
    gw = block.backward(dout, saved, p)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got, saved = block.forward(x, res, p, stream=st)
    gg = block.backward(dout, saved, p, stream=st)
    st.synchronize()
    assert torch.equal(got, want) and torch.equal(gg["x"], gw["x"]) and torch.equal(gg["up"]["A"], gw["up"]["A"])
    assert torch.equal(gg["down"]["m"], gw["down"]["m"])


def test_block_refuses_mixed_types():
    p, rng = make("bf16", 64, 64, 4)
    x = draw(rng, (8, 64), "f16")
    with pytest.raises((ValueError, TypeError)):
        block.adapted_linear(x, p.up, p.up.m)
    with pytest.raises((ValueError, TypeError)):
        bnd.dora_rms_norm(x, p.norm_weight, 1e-6, residual=draw(rng, (8, 64), "bf16"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_empty_batch_has_zero_gradients(dtype):
    p, rng = make(dtype, 64, 96, 8)
    x, dout = draw(rng, (0, 64), dtype), draw(rng, (0, 64), dtype)
    out, saved = block.forward(x, x.clone(), p)
    assert out.shape == (0, 64)
    stale = [torch.full((n,), float("nan"), device="cuda") for n in (64, 64, 96, 96, 768, 768) * 4]
    del stale
    g = block.backward(dout, saved, p)
    assert g["x"].shape == (0, 64) and (g["norm_weight"] == 0).all()
    for side in ("up", "down"):
        for k in ("A", "B", "m", "bias"):
            assert (g[side][k] == 0).all(), (side, k)
