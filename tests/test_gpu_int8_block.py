"""The feed-forward block with a layer norm, on 8-bit bases, and with packed activations, against the fp64 reference and
against itself on the values that its int8 rows stand for.

Tolerances. As in test_gpu_block.py: 1e-4 of a result's norm for fp32's chained
sums, 8 roundings of 2^-8 for bf16, 16 for gradients. A row packed with one
scale is off by at most half a step, max / 254, a value; the largest of these
normal values is at most 6 times their root mean square, so 3 / 127 of the
row's norm, once for each packing on the way.
"""

import numpy as np
import pytest
import torch

from block_helpers import draw, host, vec
from dora_weight_norm_amd import binding as bnd
from dora_weight_norm_amd import block
from oracle import int8_oracle as Q
from test_gpu_block import layer64, make, rel

pytestmark = pytest.mark.gpu
PACK = 3 / 127


def layered(p, rng, bias=True):
    """The block with a layer norm."""
    d = p.norm_weight.numel()
    return block.FeedForward(p.norm_weight, p.up, p.down, p.act, 1e-5, "layer", vec(rng, d, 0.1, 0.0) if bias else None)


def block64(x, res, p, nw=None, nb=None, up=None, down=None):
    n, h, _, _ = Q.layer_norm(x, res, host(p.norm_weight) if nw is None else nw, host(p.norm_bias) if nb is None else nb,
                              p.eps)
    a = layer64(n, p.up, p.act, **(up or {}))
    return layer64(a, p.down, residual=h, **(down or {}))


def thawed(layer):
    """The layer on the 16-bit values of its 8-bit base."""
    return block.AdaptedLayer(bnd.dora_dequantize_rows(layer.W.q, layer.W.scale, dtype=layer.A.dtype), layer.A, layer.B,
                              layer.m, layer.s, layer.bias, layer.eps)


@pytest.mark.parametrize("dtype,T,d,f,r", [("f32", 40, 64, 96, 8), ("bf16", 300, 264, 520, 24), ("f16", 1, 256, 384, 16),
                                           ("bf16", 7, 1000, 777, 5)])
@pytest.mark.parametrize("bias", [True, False])
def test_forward_with_a_layer_norm(dtype, T, d, f, r, bias):
    p, rng = make(dtype, d, f, r)
    p = layered(p, rng, bias)
    x, res = draw(rng, (T, d), dtype, 1.0, 0.5), draw(rng, (T, d), dtype)
    out, _ = block.forward(x, res, p)
    assert rel(out, block64(host(x), host(res), p)) <= (1e-4 if dtype == "f32" else 8 * 2.0 ** -8)


def test_layer_norm_block_gradients_against_differences():
    p, rng = make("f32", 48, 72, 8)
    p = layered(p, rng)
    x, res, dout = (draw(rng, (20, 48), "f32") for _ in range(3))
    _, saved = block.forward(x, res, p)
    g = block.backward(dout, saved, p)

    def loss(dx=0, dn=0, db=0, up=None, down=None):
        return (block64(host(x) + dx, host(res), p, host(p.norm_weight) + dn, host(p.norm_bias) + db, up, down)
                * host(dout)).sum()

    def check(grad, f, what):
        d, e = rng.standard_normal(grad.shape), 1e-5
        num = (f(e * d) - f(-e * d)) / (2 * e)
        assert abs((host(grad) * d).sum() - num) <= 1e-4 * np.linalg.norm(host(grad)) * np.linalg.norm(d), what

    check(g["x"], lambda v: loss(dx=v), "x")
    check(g["norm_weight"], lambda v: loss(dn=v), "norm_weight")
    check(g["norm_bias"], lambda v: loss(db=v), "norm_bias")
    for side in ("up", "down"):
        layer = getattr(p, side)
        for k in ("A", "B", "m", "bias"):
            check(g[side][k], lambda v: loss(**{side: {k: host(getattr(layer, k)) + v}}), f"{side} {k}")
    q = layered(p, rng, bias=False)
    _, saved = block.forward(x, res, q)
    assert "norm_bias" not in block.backward(dout, saved, q)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("pack", [0, 32, 64, 128, 256])
def test_packed_activations_give_the_gradients_of_their_values(pack, norm):
    """fp32: bit for bit the gradients from the same saved activations unpacked."""
    p, rng = make("f32", 264, 520, 8)
    p = layered(p, rng) if norm == "layer" else p
    x, res, dout = (draw(rng, (70, 264), "f32") for _ in range(3))
    want, full = block.forward(x, res, p)
    out, saved = block.forward(x, res, p, pack=pack)
    assert torch.equal(out, want)
    kept = [k for k, v in saved.items() if isinstance(v, bnd.Int8Rows)]
    assert kept == ["n", "up", "u_u", "u_d"]
    back = {k: bnd.dora_dequantize_rows(*v, dtype=torch.float32) if k in kept else v for k, v in saved.items()}
    for k in kept:
        assert rel(back[k], host(full[k])) <= PACK
    got, ref = block.backward(dout, saved, p), block.backward(dout, back, p)
    for k in ("x", "norm_weight"):
        assert torch.equal(got[k], ref[k]), k
    for side in ("up", "down"):
        for k in ("A", "B", "m", "bias"):
            assert torch.equal(got[side][k], ref[side][k]), (side, k)


def test_packed_bf16_gradients_follow_the_unpacked():
    p, rng = make("bf16", 256, 512, 16)
    x, res, dout = (draw(rng, (128, 256), "bf16") for _ in range(3))
    _, full = block.forward(x, res, p)
    _, saved = block.forward(x, res, p, pack=128)
    a, b = block.backward(dout, saved, p), block.backward(dout, full, p)
    # (u and the other factor of a product are each packed)
    for g, r in ((a["x"], b["x"]), (a["norm_weight"], b["norm_weight"]), (a["up"]["A"], b["up"]["A"]),
                 (a["up"]["m"], b["up"]["m"]), (a["down"]["B"], b["down"]["B"]), (a["down"]["A"], b["down"]["A"])):
        assert rel(g, host(r)) <= 2 * PACK + 16 * 2.0 ** -8
    held = sum(v.q.numel() + 4 * v.scale.numel() for v in saved.values() if isinstance(v, bnd.Int8Rows))
    assert held < 0.53 * sum(2 * full[k].numel() for k in ("n", "up", "u_u", "u_d"))


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 16), ("f16", 200)])
def test_block_on_8_bit_bases(dtype, T, norm):
    p, rng = make(dtype, 512, 1024, 16)
    p = layered(p, rng) if norm == "layer" else p
    p8 = block.FeedForward(p.norm_weight, block.int8_base(p.up), block.int8_base(p.down), p.act, p.eps, p.norm, p.norm_bias)
    p16 = block.FeedForward(p.norm_weight, thawed(p8.up), thawed(p8.down), p.act, p.eps, p.norm, p.norm_bias)
    x, res, dout = (draw(rng, (T, 512), dtype) for _ in range(3))
    g = [layer.magnitude()[1] for layer in (p8.up, p8.down)]
    for a, b in zip(g, (p16.up.magnitude()[1], p16.down.magnitude()[1])):
        assert torch.equal(a, b)
    ref, s16 = block.forward(x, res, p16)
    out, saved = block.forward(x, res, p8)
    assert rel(out, host(ref)) <= 2 * PACK + 8 * 2.0 ** -8
    assert torch.equal(block.forward_int8(x, res, p8, *g), out)
    got, want = block.backward(dout, saved, p8), block.backward(dout, s16, p16)
    for k in ("x", "norm_weight"):
        assert rel(got[k], host(want[k])) <= 4 * PACK + 16 * 2.0 ** -8, k
    for side in ("up", "down"):
        for k in ("A", "B", "m", "bias"):
            assert rel(got[side][k], host(want[side][k])) <= 4 * PACK + 16 * 2.0 ** -8, (side, k)
    # with whole rows the norm's own rows are what is kept
    _, packed = block.forward(x, res, p8, pack=0)
    again = block.backward(dout, packed, p8)
    assert rel(again["x"], host(got["x"])) <= 4 * PACK + 16 * 2.0 ** -8


@pytest.mark.parametrize("T", [1, 16, 200])
def test_8_bit_serving_with_a_layer_norm(T):
    p, rng = make("bf16", 512, 1024, 16)
    p = layered(p, rng)
    x, res = draw(rng, (T, 512), "bf16"), draw(rng, (T, 512), "bf16")
    _, g_down = p.down.magnitude()
    out = block.forward_8bit(x, res, p, block.freeze_8bit(p.up), g_down)
    assert rel(out, block64(host(x), host(res), p)) <= 2 * 2.0 ** -4 + 8 * 2.0 ** -8


def test_int8_block_on_a_stream_of_its_own_and_in_a_graph():
    p, rng = make("bf16", 256, 512, 16)
    p = layered(p, rng)
    p = block.FeedForward(p.norm_weight, block.int8_base(p.up), block.int8_base(p.down), p.act, p.eps, p.norm, p.norm_bias)
    x, res, dout = (draw(rng, (64, 256), "bf16") for _ in range(3))

    def step(**kw):
        y, saved = block.forward(x, res, p, pack=128, **kw)
        g = block.backward(dout, saved, p, **kw)
        return [y, g["x"], g["norm_weight"], g["norm_bias"], g["up"]["A"], g["down"]["m"], g["down"]["B"]]

    want = step()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = step(stream=st)
    st.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for v in got:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        eager = step()
        torch.cuda.synchronize()
        for a, b in zip(eager, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("pack", [None, 128])
def test_an_empty_batch_on_8_bit_bases(pack):
    p, rng = make("bf16", 64, 96, 8)
    p = layered(p, rng)
    p = block.FeedForward(p.norm_weight, block.int8_base(p.up), block.int8_base(p.down), p.act, p.eps, p.norm, p.norm_bias)
    x, dout = draw(rng, (0, 64), "bf16"), draw(rng, (0, 64), "bf16")
    out, saved = block.forward(x, x.clone(), p, pack=pack)
    assert out.shape == (0, 64)
    g = block.backward(dout, saved, p)
    assert g["x"].shape == (0, 64) and (g["norm_weight"] == 0).all() and (g["norm_bias"] == 0).all()
    for side in ("up", "down"):
        for k in ("A", "B", "m", "bias"):
            assert (g[side][k] == 0).all(), (side, k)


def test_int8_block_refusals():
    p, rng = make("f32", 64, 64, 4)
    x = draw(rng, (8, 64), "f32")
    with pytest.raises(TypeError):                      # the integer product's pair is of 16 bits
        block.adapted_linear(x, block.int8_base(p.up), p.up.m)
    with pytest.raises(ValueError):
        block.forward(x, x, p, pack=100)
    with pytest.raises(ValueError):
        block.FeedForward(p.norm_weight, p.up, p.down, norm="batch")
    with pytest.raises(ValueError):
        block.FeedForward(p.norm_weight, p.up, p.down, norm_bias=p.norm_weight)


def test_freezing_a_layer_on_an_8_bit_base():
    p, rng = make("bf16", 256, 384, 16)
    a, b = block.int8_base(p.up), thawed(block.int8_base(p.up))
    x, y = block.freeze_8bit(a), block.freeze_8bit(b)
    assert torch.equal(x.w.view(torch.uint8), y.w.view(torch.uint8)) and torch.equal(x.scale, y.scale)
