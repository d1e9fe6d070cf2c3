"""A feed-forward block of adapted layers on libdora's kernels.

    h   = x + residual            n = rms_norm(h) or layer_norm(h)
    up  = act(g_u * (n W_u^T + s_u (n A_u^T) B_u^T) + bias_u)
    out = h + g_d * (up W_d^T + s_d (up A_d^T) B_d^T) + bias_d

Each adapted layer is two products: t = x A^T, and the layer itself, whose
epilogue applies the magnitude, bias, activation and residual, so that
neither the base nor the low-rank projection is written to memory. The
training forward keeps what the backward reads; W is frozen and the row norm
detached, as in the DoRA write-ups, so the gradients are those of A, B, the
magnitude, the bias, the norm's weight (and bias) and the input. `freeze_8bit`
merges a layer's direction and holds it in 8 bits, for a forward whose norm
writes 8-bit rows.

    from dora_weight_norm_amd import block
    y, saved = block.forward(x, residual, p)
    grads = block.backward(dy, saved, p)

8-bit integers serve two ends, each by itself or both at once. `int8_base` holds
a layer's frozen W as int8 rows: its product is then one of integers, with the
input packed a scale a token, and the adapter beside it in 16 bits, in training
and (`forward_int8`) in serving (the row norm of such a base is that of its values in
16 bits, and every training forward writes these for it, a layer at a time:
`AdaptedLayer.magnitude`). And `forward(..., pack=128)` keeps the activations that the backward
reads (the layers' inputs and their products before the magnitude) as int8 rows
with a scale for each 128 columns, at half of their memory (h and both t = x A^T
stay as they are); the gradients are those of the values so kept.
"""

from __future__ import annotations

from dataclasses import dataclass, replace

import torch

from . import binding as bnd

__all__ = ["AdaptedLayer", "FeedForward", "adapted_linear", "adapted_linear_backward", "forward", "backward",
           "Frozen8Bit", "freeze_8bit", "forward_8bit", "int8_base", "forward_int8"]


@dataclass
class AdaptedLayer:
    """W [d_out, d_in], A [r, d_in], B [d_out, r] of one dtype; m, bias float32 [d_out]; s = alpha / r.
    W may be bnd.Int8Rows with one scale a row (A and B then of 16 bits)."""
    W: torch.Tensor | bnd.Int8Rows
    A: torch.Tensor
    B: torch.Tensor
    m: torch.Tensor
    s: float
    bias: torch.Tensor | None = None
    eps: float = 1e-6

    def weight(self, stream=None):
        """W in A's dtype: itself, or the values that its int8 rows stand for, rounded to it (a new tensor each time)."""
        if isinstance(self.W, bnd.Int8Rows):
            return bnd.dora_dequantize_rows(*self.W, dtype=self.A.dtype, stream=stream)
        return self.W

    def magnitude(self, stream=None):
        """(wnorm, g) of the layer as it stands, float32 [d_out].

        On an 8-bit W the norm is of weight(): the call brings the whole W back to A's dtype first, in memory of its
        own, and its values are rounded to 16 bits, which the integer product's are not. The two norms differ by less
        than half a step of that type times the row norm of W: 2^-8 in bf16 and, of values from 2^-14 on, 2^-11 in
        fp16 (with normally distributed W up to 1.2e-3 and 1.7e-4, for a row has 255 values at most, and equal ones
        round alike). Training and serving take the same g."""
        return bnd.dora_factored_norm(self.weight(stream), self.A, self.B, self.s, m=self.m, eps=self.eps,
                                      stream=stream)


@dataclass
class FeedForward:
    norm_weight: torch.Tensor   # float32 [d_in]
    up: AdaptedLayer
    down: AdaptedLayer
    act: str = "silu"
    eps: float = 1e-6
    norm: str = "rms"                       # or "layer"
    norm_bias: torch.Tensor | None = None   # float32 [d_in], the layer norm's

    def __post_init__(self):
        if self.norm not in ("rms", "layer"):
            raise ValueError(f"norm must be rms or layer, got {self.norm!r}")
        if self.norm == "rms" and self.norm_bias is not None:
            raise ValueError("the RMS norm has no bias")


def _packed(x, group, stream):
    return bnd.Int8Rows(*bnd.dora_quantize_rows(x, group=group, stream=stream), group)


def adapted_linear(x, layer: AdaptedLayer, g, act: str = "none", residual=None, save: bool = False, stream=None,
                   rows: bnd.Int8Rows | None = None):
    """act(g * (x W^T + s (x A^T) B^T) + bias) + residual. Returns (y, t, u): t = x A^T, and u, the product before
    the magnitude, if `save` (else None). On an 8-bit W the product is of integers; `rows` is x packed with one scale
    a row, where the caller has it (else it is packed here)."""
    t, _ = bnd.dora_matmul(x, layer.A, stream=stream)
    if isinstance(layer.W, bnd.Int8Rows):
        rows = _packed(x, 0, stream) if rows is None else rows
        y, u = bnd.dora_matmul_int8(rows.q, layer.W.q, rows.scale, layer.W.scale, col_scale=g, t=t, b=layer.B,
                                    s=layer.s, bias=layer.bias, act=act, residual=residual, out_dtype=x.dtype,
                                    save=save, stream=stream)
        return y, t, u
    y, u = bnd.dora_matmul(x, layer.W, col_scale=g, t=t, b=layer.B, s=layer.s, bias=layer.bias, act=act,
                           residual=residual, save=save, stream=stream)
    return y, t, u


def _matmul_backward(dy, u, x, w, **kw):
    held = any(isinstance(v, bnd.Int8Rows) for v in (u, x, w))
    return (bnd.dora_matmul_backward_int8 if held else bnd.dora_matmul_backward)(dy, u, x, w, **kw)


def adapted_linear_backward(dy, u, t, x, layer: AdaptedLayer, g, act: str = "none", stream=None):
    """Gradients of adapted_linear: a dict with x, A, B (storage dtype), g and bias (float32 [d_out]); the
    residual's is dy. W is frozen. u and x may be Int8Rows. On an 8-bit W the packing of x for its product counts as
    the identity.

    The products take no scale or addend, so s is applied to dA, dB and the adapter's part of dx after they are
    rounded, which rounds each a second time, and dx is rounded once more as their sum."""
    dx, _, dbias, dg, du = _matmul_backward(dy, u, None, layer.W, col_scale=g, bias=layer.bias, act=act,
                                            need_dw=False, need_dbias=layer.bias is not None, stream=stream)
    plain = dict(need_dbias=False, need_dcol_scale=False, stream=stream)
    dt, dB, _, _, _ = bnd.dora_matmul_backward(du, du, t, layer.B, **plain)
    dx2, dA, _, _, _ = _matmul_backward(dt, dt, x, layer.A, **plain)
    with bnd._on(stream):
        return {"x": dx.add_(dx2, alpha=layer.s), "A": dA.mul_(layer.s), "B": dB.mul_(layer.s), "g": dg,
                "bias": dbias}


def _norm(x, residual, p: FeedForward, stream, stats=True):
    """(n, h, mean, rstd, rows): mean for the layer norm alone; rows, n as int8 rows, where the up projection is one
    of integers (the layer norm writes them beside n)."""
    int8 = isinstance(p.up.W, bnd.Int8Rows)
    if p.norm == "rms":
        n, h, rstd = bnd.dora_rms_norm(x, p.norm_weight, p.eps, residual=residual, want_rstd=stats, stream=stream)
        return n, h, None, rstd, _packed(n, 0, stream) if int8 else None
    if not int8:
        n, h, mean, rstd = bnd.dora_layer_norm(x, p.norm_weight, p.norm_bias, p.eps, residual=residual,
                                               want_stats=stats, stream=stream)
        return n, h, mean, rstd, None
    with bnd._on(stream):
        n = torch.empty_like(x)
    q, scale, h, mean, rstd = bnd.dora_layer_norm_quant(x, p.norm_weight, p.norm_bias, p.eps, residual=residual, y=n,
                                                        want_stats=stats, stream=stream)
    return n, h, mean, rstd, bnd.Int8Rows(q, scale)


def forward(x, residual, p: FeedForward, stream=None, pack: int | None = None):
    """Training forward on x, residual [T, d]. Returns (out, saved); out is the next residual stream. `pack`: the
    layers' inputs and products are saved as int8 rows with a scale for each `pack` columns (32, 64, 128 or 256; 0:
    for each row)."""
    n, h, mean, rstd, rows = _norm(x, residual, p, stream)
    wn_u, g_u = p.up.magnitude(stream)
    up, t_u, u_u = adapted_linear(n, p.up, g_u, act=p.act, save=True, stream=stream, rows=rows)
    wn_d, g_d = p.down.magnitude(stream)
    up_rows = _packed(up, 0, stream) if isinstance(p.down.W, bnd.Int8Rows) else None
    out, t_d, u_d = adapted_linear(up, p.down, g_d, residual=h, save=True, stream=stream, rows=up_rows)
    if pack is not None:
        n = rows if pack == 0 and rows is not None else _packed(n, pack, stream)
        up = up_rows if pack == 0 and up_rows is not None else _packed(up, pack, stream)
        u_u, u_d = _packed(u_u, pack, stream), _packed(u_d, pack, stream)
    return out, dict(n=n, h=h, mean=mean, rstd=rstd, wn_u=wn_u, g_u=g_u, up=up, t_u=t_u, u_u=u_u, wn_d=wn_d, g_d=g_d,
                     t_d=t_d, u_d=u_d)


def backward(dout, saved: dict, p: FeedForward, stream=None):
    """Gradients of forward: a dict with x (and, the same, residual), norm_weight (and norm_bias with the layer norm),
    and for each of up and down a dict with A, B, m and bias."""
    v = saved
    down = adapted_linear_backward(dout, v["u_d"], v["t_d"], v["up"], p.down, v["g_d"], stream=stream)
    up = adapted_linear_backward(down.pop("x"), v["u_u"], v["t_u"], v["n"], p.up, v["g_u"], act=p.act, stream=stream)
    grads = {"up": up, "down": down}
    if p.norm == "layer":
        need = p.norm_bias is not None
        grads["x"], grads["norm_weight"], db = bnd.dora_layer_norm_backward(
            up.pop("x"), v["h"], v["mean"], v["rstd"], p.norm_weight, dh=dout, need_dbias=need, stream=stream)
        if need:
            grads["norm_bias"] = db
    else:
        grads["x"], grads["norm_weight"] = bnd.dora_rms_norm_backward(up.pop("x"), v["h"], v["rstd"], p.norm_weight,
                                                                      dh=dout, stream=stream)
    with bnd._on(stream):
        for side, layer, wn in ((up, p.up, v["wn_u"]), (down, p.down, v["wn_d"])):
            side["m"] = side.pop("g") / wn.clamp(min=layer.eps)   # g = m / max(wnorm, eps)
    return grads


def int8_base(layer: AdaptedLayer, stream=None) -> AdaptedLayer:
    """The layer on its frozen W in 8-bit integers with one scale a row; the adapter, magnitude and bias are shared."""
    return replace(layer, W=_packed(layer.W, 0, stream))


def forward_int8(x, residual, p: FeedForward, g_up, g_down, stream=None):
    """Serving forward on 8-bit bases with unmerged adapters (g_up, g_down: the layers' magnitude scales, computed
    once). Returns the next residual stream."""
    n, h, _, _, rows = _norm(x, residual, p, stream, stats=False)
    a, _, _ = adapted_linear(n, p.up, g_up, act=p.act, stream=stream, rows=rows)
    return adapted_linear(a, p.down, g_down, residual=h, stream=stream)[0]


@dataclass
class Frozen8Bit:
    """A layer's direction W + s B A in 8 bits: w float8_e4m3fn [d_out, d_in]; scale = g times the rows' scales."""
    w: torch.Tensor
    scale: torch.Tensor
    bias: torch.Tensor | None


def freeze_8bit(layer: AdaptedLayer, stream=None) -> Frozen8Bit:
    """Merges and quantises a layer once, when serving starts."""
    _, g = layer.magnitude(stream)
    W = layer.weight(stream)
    with bnd._on(stream):
        v = W.float() + layer.s * (layer.B.float() @ layer.A.float())
        scale = (v.abs().amax(1) / 448.0).clamp(min=2.0 ** -100)
        return Frozen8Bit((v / scale[:, None]).to(torch.float8_e4m3fn), scale * g, layer.bias)


def forward_8bit(x, residual, p: FeedForward, up: Frozen8Bit, g_down, stream=None):
    """Serving forward: the norm writes 8-bit rows, the up projection runs in 8 bits, the down projection is the
    adapted layer itself (g_down: its magnitude scale). Returns the next residual stream."""
    if p.norm == "layer":
        q, scale, h, _, _ = bnd.dora_layer_norm_quant(x, p.norm_weight, p.norm_bias, p.eps, q_dtype=torch.float8_e4m3fn,
                                                      residual=residual, want_stats=False, stream=stream)
    else:
        q, scale, h, _ = bnd.dora_rms_norm_quant(x, p.norm_weight, p.eps, residual=residual, want_rstd=False,
                                                 stream=stream)
    a, _ = bnd.dora_matmul(q, up.w, row_scale=scale, col_scale=up.scale, bias=up.bias, act=p.act, out_dtype=x.dtype,
                           stream=stream)
    return adapted_linear(a, p.down, g_down, residual=h, stream=stream)[0]
