"""A feed-forward block of adapted layers on libdora's kernels.

    h   = x + residual            n = rms_norm(h)
    up  = act(g_u * (n W_u^T + s_u (n A_u^T) B_u^T) + bias_u)
    out = h + g_d * (up W_d^T + s_d (up A_d^T) B_d^T) + bias_d

Each adapted layer is two products: t = x A^T, and the layer itself, whose
epilogue applies the magnitude, bias, activation and residual, so that
neither the base nor the low-rank projection is written to memory. The
training forward keeps what the backward reads; W is frozen and the row norm
detached, as in the DoRA write-ups, so the gradients are those of A, B, the
magnitude, the bias, the norm's weight and the input. `freeze_8bit` merges a
layer's direction and holds it in 8 bits, for a forward whose norm writes 8-bit
rows.

    from dora_weight_norm_amd import block
    y, saved = block.forward(x, residual, p)
    grads = block.backward(dy, saved, p)
"""

from __future__ import annotations

from dataclasses import dataclass

import torch

from . import binding as bnd

__all__ = ["AdaptedLayer", "FeedForward", "adapted_linear", "adapted_linear_backward", "forward", "backward",
           "Frozen8Bit", "freeze_8bit", "forward_8bit"]


@dataclass
class AdaptedLayer:
    """W [d_out, d_in], A [r, d_in], B [d_out, r] of one dtype; m, bias float32 [d_out]; s = alpha / r."""
    W: torch.Tensor
    A: torch.Tensor
    B: torch.Tensor
    m: torch.Tensor
    s: float
    bias: torch.Tensor | None = None
    eps: float = 1e-6

    def magnitude(self, stream=None):
        """(wnorm, g) of the layer as it stands, float32 [d_out]."""
        return bnd.dora_factored_norm(self.W, self.A, self.B, self.s, m=self.m, eps=self.eps, stream=stream)


@dataclass
class FeedForward:
    norm_weight: torch.Tensor   # float32 [d_in]
    up: AdaptedLayer
    down: AdaptedLayer
    act: str = "silu"
    eps: float = 1e-6


def adapted_linear(x, layer: AdaptedLayer, g, act: str = "none", residual=None, save: bool = False, stream=None):
    """act(g * (x W^T + s (x A^T) B^T) + bias) + residual. Returns (y, t, u): t = x A^T, and u, the product before
    the magnitude, if `save` (else None)."""
    t, _ = bnd.dora_matmul(x, layer.A, stream=stream)
    y, u = bnd.dora_matmul(x, layer.W, col_scale=g, t=t, b=layer.B, s=layer.s, bias=layer.bias, act=act,
                           residual=residual, save=save, stream=stream)
    return y, t, u


def adapted_linear_backward(dy, u, t, x, layer: AdaptedLayer, g, act: str = "none", stream=None):
    """Gradients of adapted_linear: a dict with x, A, B (storage dtype), g and bias (float32 [d_out]); the
    residual's is dy. W is frozen.

    The products take no scale or addend, so s is applied to dA, dB and the adapter's part of dx after they are
    rounded, which rounds each a second time, and dx is rounded once more as their sum."""
    dx, _, dbias, dg, du = bnd.dora_matmul_backward(dy, u, None, layer.W, col_scale=g, bias=layer.bias, act=act,
                                                    need_dw=False, need_dbias=layer.bias is not None, stream=stream)
    plain = dict(need_dbias=False, need_dcol_scale=False, stream=stream)
    dt, dB, _, _, _ = bnd.dora_matmul_backward(du, du, t, layer.B, **plain)
    dx2, dA, _, _, _ = bnd.dora_matmul_backward(dt, dt, x, layer.A, **plain)
    with bnd._on(stream):
        return {"x": dx.add_(dx2, alpha=layer.s), "A": dA.mul_(layer.s), "B": dB.mul_(layer.s), "g": dg,
                "bias": dbias}


def forward(x, residual, p: FeedForward, stream=None):
    """Training forward on x, residual [T, d]. Returns (out, saved); out is the next residual stream."""
    n, h, rstd = bnd.dora_rms_norm(x, p.norm_weight, p.eps, residual=residual, stream=stream)
    wn_u, g_u = p.up.magnitude(stream)
    up, t_u, u_u = adapted_linear(n, p.up, g_u, act=p.act, save=True, stream=stream)
    wn_d, g_d = p.down.magnitude(stream)
    out, t_d, u_d = adapted_linear(up, p.down, g_d, residual=h, save=True, stream=stream)
    return out, dict(n=n, h=h, rstd=rstd, wn_u=wn_u, g_u=g_u, up=up, t_u=t_u, u_u=u_u, wn_d=wn_d, g_d=g_d, t_d=t_d,
                     u_d=u_d)


def backward(dout, saved: dict, p: FeedForward, stream=None):
    """Gradients of forward: a dict with x (and, the same, residual), norm_weight, and for each of up and down a
    dict with A, B, m and bias."""
    v = saved
    down = adapted_linear_backward(dout, v["u_d"], v["t_d"], v["up"], p.down, v["g_d"], stream=stream)
    up = adapted_linear_backward(down.pop("x"), v["u_u"], v["t_u"], v["n"], p.up, v["g_u"], act=p.act, stream=stream)
    dx, dw = bnd.dora_rms_norm_backward(up.pop("x"), v["h"], v["rstd"], p.norm_weight, dh=dout, stream=stream)
    with bnd._on(stream):
        for grads, layer, wn in ((up, p.up, v["wn_u"]), (down, p.down, v["wn_d"])):
            grads["m"] = grads.pop("g") / wn.clamp(min=layer.eps)   # g = m / max(wnorm, eps)
    return {"x": dx, "norm_weight": dw, "up": up, "down": down}


@dataclass
class Frozen8Bit:
    """A layer's direction W + s B A in 8 bits: w float8_e4m3fn [d_out, d_in]; scale = g times the rows' scales."""
    w: torch.Tensor
    scale: torch.Tensor
    bias: torch.Tensor | None


def freeze_8bit(layer: AdaptedLayer, stream=None) -> Frozen8Bit:
    """Merges and quantises a layer once, when serving starts."""
    _, g = layer.magnitude(stream)
    with bnd._on(stream):
        v = layer.W.float() + layer.s * (layer.B.float() @ layer.A.float())
        scale = (v.abs().amax(1) / 448.0).clamp(min=2.0 ** -100)
        return Frozen8Bit((v / scale[:, None]).to(torch.float8_e4m3fn), scale * g, layer.bias)


def forward_8bit(x, residual, p: FeedForward, up: Frozen8Bit, g_down, stream=None):
    """Serving forward: the norm writes 8-bit rows, the up projection runs in 8 bits, the down projection is the
    adapted layer itself (g_down: its magnitude scale). Returns the next residual stream."""
    q, scale, h, _ = bnd.dora_rms_norm_quant(x, p.norm_weight, p.eps, residual=residual, want_rstd=False,
                                             stream=stream)
    a, _ = bnd.dora_matmul(q, up.w, row_scale=scale, col_scale=up.scale, bias=up.bias, act=p.act, out_dtype=x.dtype,
                           stream=stream)
    return adapted_linear(a, p.down, g_down, residual=h, stream=stream)[0]
