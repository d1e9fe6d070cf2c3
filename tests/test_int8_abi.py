"""Argument errors and workspace queries of the layer norm, of int8 rows and of the integer product (no GPU: every call
returns before a launch)."""

import ctypes
import os

import pytest
import torch

from dora_weight_norm_amd import binding as bnd

pytestmark = pytest.mark.skipif(not os.path.exists(bnd.LIB_PATH), reason="libdora.so not built")
P = ctypes.c_void_p


def _norm(x=0x100000, residual=0x200000, weight=0x300000, bias=0x310000, eps=1e-6, dtype=0, T=4, d=32, h=0x400000,
          y=0x500000, q=None, q_dtype=0, scale=None, mean=0x610000, rstd=0x600000):
    return bnd.load().dora_layer_norm(P(x), P(residual), P(weight), P(bias), eps, dtype, T, d, P(h), P(y), P(q), q_dtype,
                                      P(scale), P(mean), P(rstd), None)


def test_layer_norm_refusals():
    assert _norm(dtype=3) == 2 and _norm(dtype=4) == 2
    assert _norm(q=0x700000, scale=0x710000, q_dtype=0) == 2 and _norm(q=0x700000, scale=0x710000, q_dtype=5) == 2
    assert _norm(T=-1) == 1 and _norm(d=-1) == 1 and _norm(T=1 << 31) == 1 and _norm(T=1 << 20, d=1 << 20) == 1
    assert _norm(eps=0.0) == 1 and _norm(eps=float("nan")) == 1 and _norm(eps=float("inf")) == 1
    assert _norm(x=None) == 1 and _norm(y=None) == 1
    assert _norm(q=0x700000, q_dtype=4) == 1 and _norm(scale=0x700000) == 1      # one without the other
    assert _norm(residual=None) == 1                                              # h without a residual
    assert _norm(x=0x100001) == 1 and _norm(mean=0x610002) == 1 and _norm(bias=0x310001) == 1
    assert _norm(y=0x100000) == 1 and _norm(h=0x100010) == 1 and _norm(mean=0x600004) == 1
    assert _norm(mean=0x310000) == 1                                              # over the bias
    assert _norm(q=0x500010, q_dtype=4, scale=0x710000) == 1                      # over y
    assert _norm(T=0) == 0
    assert _norm(d=0) == 1 and _norm(d=0, rstd=None) == 1 and _norm(d=0, rstd=None, mean=None) == 0


def _norm_bwd(dy=0x100000, dh=0x200000, h=0x300000, mean=0x410000, rstd=0x400000, weight=0x500000, dtype=0, T=4, d=32,
              dx=0x600000, dweight=0x700000, dbias=0x710000, ws=0x800000, ws_bytes=1 << 20):
    return bnd.load().dora_layer_norm_backward(P(dy), P(dh), P(h), P(mean), P(rstd), P(weight), dtype, T, d, P(dx),
                                               P(dweight), P(dbias), P(ws), ws_bytes, None)


def test_layer_norm_backward_refusals():
    assert _norm_bwd(dtype=3) == 2 and _norm_bwd(T=-1) == 1
    for k in ("dy", "h", "mean", "rstd", "dx"):
        assert _norm_bwd(**{k: None}) == 1, k
    assert _norm_bwd(dx=0x300000) == 1 and _norm_bwd(dx=0x100010) == 1 and _norm_bwd(dbias=0x700004) == 1
    assert _norm_bwd(ws=None) == 4 and _norm_bwd(ws_bytes=8) == 4 and _norm_bwd(ws=0x800010) == 4
    assert _norm_bwd(ws=None, dweight=None) == 4                # dbias alone needs it too
    assert _norm_bwd(ws=0x100000) == 1 and _norm_bwd(d=0) == 0
    sz = ctypes.c_size_t()
    f = bnd.load().dora_layer_norm_backward_workspace_size
    assert f(4, 32, 0, ctypes.byref(sz)) == 0 and sz.value == 4 * 2 * 32 * 4
    assert f(4, 32, 0, None) == 1 and f(4, 32, 3, ctypes.byref(sz)) == 2 and f(-1, 32, 0, ctypes.byref(sz)) == 1


def _quant(x=0x100000, dtype=0, T=4, d=64, group=0, q=0x200000, scale=0x300000):
    return bnd.load().dora_quantize_rows(P(x), dtype, T, d, group, P(q), P(scale), None)


def _dequant(q=0x200000, scale=0x300000, T=4, d=64, group=0, dtype=0, x=0x100000):
    return bnd.load().dora_dequantize_rows(P(q), P(scale), T, d, group, dtype, P(x), None)


def test_int8_rows_refusals():
    for f in (_quant, _dequant):
        assert f(dtype=3) == 2 and f(dtype=4) == 2
        assert f(T=-1) == 1 and f(d=-1) == 1 and f(T=1 << 20, d=1 << 20) == 1
        for g in (-1, 1, 16, 48, 96, 512):
            assert f(group=g) == 1, g
        assert f(x=None) == 1 and f(q=None) == 1 and f(scale=None) == 1
        assert f(x=0x100001) == 1 and f(scale=0x300002) == 1
        assert f(q=0x100010) == 1 and f(scale=0x100010) == 1
        assert f(T=0) == 0 and f(d=0, group=32) == 0
    assert _quant(scale=0x200010) == 1
    assert _quant(d=0) == 1                                     # a row of nothing has no scale
    assert _dequant(d=0) == 0


def _mm(x=0x1000000, row_scale=0x2800000, w=0x2000000, w_scale=0x2900000, M=4, N=32, K=64, col_scale=0x3000000, t=None,
        b=None, r=0, s=1.0, bias=0x4000000, act=0, residual=None, out_dtype=0, y=0x5000000, u=None, ws=0x8000000,
        ws_bytes=1 << 24):
    return bnd.load().dora_matmul_int8(P(x), P(row_scale), P(w), P(w_scale), M, N, K, P(col_scale), P(t), P(b), r, s,
                                       P(bias), act, P(residual), out_dtype, P(y), P(u), P(ws), ws_bytes, None)


def test_int8_product_refusals():
    pair = dict(r=8, t=0x6000000, b=0x7000000)
    assert _mm(out_dtype=3) == 2 and _mm(out_dtype=4) == 2
    assert _mm(M=-1) == 1 and _mm(N=-1) == 1 and _mm(K=-1) == 1 and _mm(r=-1) == 1
    assert _mm(K=131072) == 1 and _mm(M=1 << 30) == 1 and _mm(M=4, N=1 << 23) == 1
    assert _mm(M=1 << 20, N=1 << 14) == 1
    assert _mm(act=5) == 1 and _mm(act=-1) == 1
    assert _mm(s=float("nan")) == 1 and _mm(s=float("inf")) == 1
    for s in (2.0 ** -65, -2.0 ** -65, 2.0 ** 65, 1e-40):
        assert _mm(**pair, s=s) == 1, s
    assert _mm(**pair, out_dtype=1) == 1                        # no pair with fp32 outputs
    for k in ("x", "w", "y", "row_scale", "w_scale"):
        assert _mm(**{k: None}) == 1, k
    assert _mm(r=8) == 1 and _mm(r=8, t=0x6000000) == 1
    assert _mm(**{**pair, "t": 0x6000001}) == 1 and _mm(bias=0x4000002) == 1 and _mm(w_scale=0x2900002) == 1
    assert _mm(y=0x1000000) == 1 and _mm(y=0x2000010) == 1 and _mm(y=0x2800000) == 1 and _mm(u=0x2900000) == 1
    assert _mm(residual=0x5000010) == 1 and _mm(u=0x5000000) == 1
    assert _mm(M=40, K=15, ws_bytes=64) == 4 and _mm(M=40, K=15, ws=None) == 4 and _mm(M=40, K=15, ws=0x8000010) == 4
    assert _mm(M=40, K=15, ws=0x2000000) == 1 and _mm(M=40, K=15, ws=0x2800000) == 1
    assert _mm(M=0) == 0 and _mm(N=0) == 0


def test_int8_product_plans():
    def plan(*a, **k):
        p = bnd.dora_matmul_int8_plan_info(*a, **k)
        return p["tile_rows"], p["splits"] > 1, p["copies"], p["few_rows"]

    assert plan(8192, 8192, 8192, 384) == (256, False, 0, -1)
    assert plan(1, 8192, 8192, 384)[0] == 0 and plan(1, 8192, 8192, 384)[3] == 8
    assert plan(16, 28672, 8192, 0)[3] == 16 and plan(300, 520, 264, 0)[0] == 64
    assert plan(32, 28672, 8192, 0)[0] == 64 and plan(17, 8192, 8192, 384)[0] == 64 and plan(16, 28672, 1024, 0)[0] == 64
    assert plan(16, 8192, 28672, 0)[0] == 64 and plan(12, 8192, 28672, 0)[3] == 16 and plan(16, 8192, 16384, 0)[3] == 16
    assert plan(32, 28672, 8189, 0)[3] == 32 and plan(32, 1024, 4096, 0)[3] == 16 and plan(16, 8192, 1024, 0)[3] == 16
    # rows of no whole 16-byte chunks: x and w in bytes, the pair in 16 bits
    assert plan(3330, 2001, 776, 24)[2] == 3 and plan(3330, 2001, 784, 20)[2] == 12
    assert plan(3330, 2001, 784, 24, aligned_operands=11)[2] == 4
    # ... unless small tiles take them as they are
    for a in ((333, 1001, 776, 24), (333, 1001, 784, 20), (64, 8192, 8189, 0), (128, 8192, 512, 390)):
        assert plan(*a)[0] == 64 and plan(*a)[2] == 0
    assert plan(333, 1001, 784, 24, aligned_operands=11)[2] == 0
    assert plan(1000, 1700, 8190, 0)[2] == 3 and plan(1000, 1000, 4000, 13)[2] == 12
    assert plan(333, 1001, 15, 0)[2] == 3 and plan(333, 1001, 784, 7)[2] == 12
    assert bnd.dora_matmul_int8_plan_info(0, 8, 8, 0)["tile_rows"] == -1
    assert bnd.dora_matmul_int8_workspace_size(4096, 4096, 4095, 0) >= 2 * 4096 * 4096
    sz = ctypes.c_size_t()
    f = bnd.load().dora_matmul_int8_workspace_size
    assert f(4, 4, 131072, 0, 15, ctypes.byref(sz)) == 1 and f(4, 4, 131071, 0, 15, ctypes.byref(sz)) == 0
    assert f(4, 4, 4, 0, 15, None) == 1
    # a workspace for operands at any address serves them at all
    for M, N, K, r in ((333, 1001, 776, 24), (1000, 1000, 4000, 13), (64, 8192, 8192, 13), (100, 2000, 3008, 16),
                       (1000, 1700, 8190, 0), (1000, 1700, 8192, 5), (3330, 2001, 784, 20), (333, 1001, 15, 7)):
        sizes = [bnd.dora_matmul_int8_workspace_size(M, N, K, r, al) for al in range(16)]
        assert max(sizes) == sizes[0], (M, N, K, r)
    # a call whose s is 0 needs no more than the query with the pair says
    for M, N, K, r in ((40, 300, 63, 5), (300, 520, 4104, 700), (1000, 1000, 100, 64),
                       (32, 8192, 8192, 20), (17, 4096, 14336, 5), (1, 28672, 2048, 7), (32, 28672, 512, 600),
                       (16, 8192, 24576, 9), (64, 8192, 8192, 13), (1000, 1000, 4000, 13), (333, 1001, 777, 7)):
        assert bnd.dora_matmul_int8_workspace_size(M, N, K, 0) <= bnd.dora_matmul_int8_workspace_size(M, N, K, r)


def _rows(q=0x2000000, scale=0x2800000, group=0):
    return ctypes.byref(bnd._Int8RowsArg(q, scale, group))


def _bwd(dy=0x1000000, u=None, u8=None, x=0x3000000, x8=None, w=0x4000000, w8=None, dtype=0, M=4, N=32, K=64,
         row_scale=None, col_scale=None, bias=None, act=0, du=None, dx=0x5000000, dw=0x6000000, dbias=0x7000000,
         dcol=0x7100000, ws=0x8000000, ws_bytes=1 << 24):
    return bnd.load().dora_matmul_backward_int8(P(dy), P(u), u8, P(x), x8, P(w), w8, dtype, M, N, K, P(row_scale),
                                                P(col_scale), P(bias), act, P(du), P(dx), P(dw), P(dbias), P(dcol),
                                                P(ws), ws_bytes, None)


def test_int8_backward_refusals():
    u8 = _rows()
    assert _bwd(u8=u8, dtype=3) == 2 and _bwd(u8=u8, M=-1) == 1 and _bwd(u8=u8, act=9) == 1
    assert _bwd() == 1 and _bwd(u8=u8, u=0x2000000) == 1        # neither form of u, and both
    assert _bwd(u8=u8, x=None) == 1 and _bwd(u8=u8, w=None) == 1
    assert _bwd(u8=u8, x8=_rows(0x3100000, 0x3200000)) == 1 and _bwd(u8=u8, w8=_rows(0x4100000, 0x4200000)) == 1
    assert _bwd(u8=_rows(q=None)) == 1 and _bwd(u8=_rows(scale=None)) == 1
    assert _bwd(u8=_rows(group=48)) == 1 and _bwd(u8=u8, x=None, x8=_rows(0x3000000, 0x3200000, 1)) == 1
    assert _bwd(u8=_rows(scale=0x2800002)) == 1
    assert _bwd(u8=u8, dx=0x2000010) == 1 and _bwd(u8=u8, dbias=0x2800000) == 1
    assert _bwd(u8=u8, x=None, x8=_rows(0x6000000, 0x3200000)) == 1     # dw over x8
    assert _bwd(u8=u8, w=None, w8=_rows(0x4000000, 0x8000000)) == 1     # its scales in the workspace
    assert _bwd(u8=u8, ws=None) == 4 and _bwd(u8=u8, ws_bytes=16) == 4 and _bwd(u8=u8, dy=None) == 1
    sz = ctypes.c_size_t()
    f = bnd.load().dora_matmul_backward_int8_workspace_size
    assert f(4, 32, 64, 0, 31, 4, ctypes.byref(sz)) == 1 and f(4, 32, 64, 0, 32, 0, ctypes.byref(sz)) == 1
    assert f(4, 32, 64, 4, 31, 0, ctypes.byref(sz)) == 2 and f(4, 32, 64, 0, 31, 3, None) == 1
    assert bnd.dora_matmul_backward_int8_workspace_size(64, 64, 64, "bf16", 31, 0) == \
        bnd.dora_matmul_backward_workspace_size(64, 64, 64, "bf16", 31)


def test_binding_refuses_host_tensors_and_wrong_groups():
    x = torch.zeros(4, 8)
    for call in (lambda: bnd.dora_layer_norm(x, None, None, 1e-6), lambda: bnd.dora_quantize_rows(x),
                 lambda: bnd.dora_dequantize_rows(x.to(torch.int8), x[:, 0]),
                 lambda: bnd.dora_matmul_int8(x.to(torch.int8), x.to(torch.int8), x[:, 0], x[:, 0]),
                 lambda: bnd.dora_matmul_backward_int8(x, x, x, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        bnd.dora_matmul_int8(None, x, x, x)
    for g in (1, 33, 512, None, "128"):
        with pytest.raises(ValueError):
            bnd._scale_shape(4, 8, g)
    assert bnd._scale_shape(4, 200, 128) == (4, 2) and bnd._scale_shape(4, 200, 0) == (4,)
