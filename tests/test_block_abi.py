"""Argument errors and workspace queries of the norm and the product (no GPU: every call returns before a launch)."""

import ctypes
import os

import pytest
import torch

from dora_weight_norm_amd import binding as bnd

pytestmark = pytest.mark.skipif(not os.path.exists(bnd.LIB_PATH), reason="libdora.so not built")
P = ctypes.c_void_p


def _norm(x=0x100000, residual=0x200000, weight=0x300000, eps=1e-6, dtype=0, T=4, d=32, h=0x400000, y=0x500000,
          q=None, scale=None, rstd=0x600000):
    return bnd.load().dora_rms_norm(P(x), P(residual), P(weight), eps, dtype, T, d, P(h), P(y), P(q), P(scale),
                                    P(rstd), None)


def test_norm_refusals():
    assert _norm(dtype=3) == 2 and _norm(dtype=-1) == 2
    assert _norm(T=-1) == 1 and _norm(d=-1) == 1
    assert _norm(T=1 << 31) == 1 and _norm(T=1 << 20, d=1 << 20) == 1
    assert _norm(eps=0.0) == 1 and _norm(eps=float("nan")) == 1 and _norm(eps=float("inf")) == 1
    assert _norm(x=None) == 1
    assert _norm(y=None) == 1                                   # no output
    assert _norm(q=0x700000) == 1 and _norm(scale=0x700000) == 1   # one without the other
    assert _norm(residual=None) == 1                            # h without a residual
    assert _norm(x=0x100001) == 1 and _norm(rstd=0x600002) == 1 and _norm(weight=0x300001) == 1
    assert _norm(y=0x100010) == 1 and _norm(y=0x100000) == 1    # output over x
    assert _norm(h=0x100010) == 1                               # h partly over x
    assert _norm(h=0x500010) == 1                               # outputs overlap
    assert _norm(T=0) == 0
    assert _norm(d=0) == 1 and _norm(d=0, rstd=None) == 0


def _norm_bwd(dy=0x100000, dh=0x200000, h=0x300000, rstd=0x400000, weight=0x500000, dtype=0, T=4, d=32, dx=0x600000,
              dweight=0x700000, ws=0x800000, ws_bytes=1 << 20):
    return bnd.load().dora_rms_norm_backward(P(dy), P(dh), P(h), P(rstd), P(weight), dtype, T, d, P(dx), P(dweight),
                                             P(ws), ws_bytes, None)


def test_norm_backward_refusals():
    assert _norm_bwd(dtype=3) == 2
    assert _norm_bwd(T=-1) == 1
    assert _norm_bwd(dy=None) == 1 and _norm_bwd(h=None) == 1 and _norm_bwd(rstd=None) == 1 and _norm_bwd(dx=None) == 1
    assert _norm_bwd(dx=0x300000) == 1                          # over h
    assert _norm_bwd(dx=0x100010) == 1                          # partly over dy
    assert _norm_bwd(dweight=0x600004) == 1
    assert _norm_bwd(ws=None) == 4 and _norm_bwd(ws_bytes=8) == 4 and _norm_bwd(ws=0x800010) == 4
    assert _norm_bwd(ws=0x100000) == 1
    assert _norm_bwd(d=0) == 0
    sz = ctypes.c_size_t()
    f = bnd.load().dora_rms_norm_backward_workspace_size
    assert f(4, 32, 0, ctypes.byref(sz)) == 0 and sz.value == 4 * 32 * 4
    assert f(4, 32, 0, None) == 1 and f(4, 32, 3, ctypes.byref(sz)) == 2 and f(-1, 32, 0, ctypes.byref(sz)) == 1


def _mm(x=0x1000000, w=0x2000000, dtype=0, M=4, N=32, K=64, row_scale=None, col_scale=0x3000000, t=None, b=None, r=0,
        s=1.0, bias=0x4000000, act=0, residual=None, out_dtype=0, y=0x5000000, u=None, ws=0x8000000, ws_bytes=1 << 24):
    return bnd.load().dora_matmul(P(x), P(w), dtype, M, N, K, P(row_scale), P(col_scale), P(t), P(b), r, s, P(bias),
                                  act, P(residual), out_dtype, P(y), P(u), P(ws), ws_bytes, None)


def test_matmul_refusals():
    assert _mm(dtype=4) == 2 and _mm(out_dtype=3) == 2 and _mm(dtype=0, out_dtype=1) == 2
    assert _mm(M=-1) == 1 and _mm(N=-1) == 1 and _mm(K=-1) == 1 and _mm(r=-1) == 1
    assert _mm(K=1 << 22) == 1                                  # a row of 2^23 bytes
    assert _mm(M=1 << 30, N=1 << 10) == 1
    assert _mm(act=5) == 1 and _mm(act=-1) == 1
    assert _mm(s=float("nan")) == 1
    assert _mm(x=None) == 1 and _mm(w=None) == 1 and _mm(y=None) == 1
    assert _mm(r=8) == 1 and _mm(r=8, t=0x6000000) == 1         # the pair's operands are missing
    assert _mm(dtype=3, r=8, t=0x6000000, b=0x7000000) == 1     # no pair in e4m3
    assert _mm(x=0x1000001) == 1 and _mm(bias=0x4000002) == 1
    assert _mm(y=0x1000000) == 1 and _mm(y=0x2000010) == 1
    assert _mm(residual=0x5000010) == 1                         # partly over y
    assert _mm(u=0x5000000) == 1                                # u over y
    assert _mm(M=40, K=63, ws_bytes=64) == 4 and _mm(M=40, K=63, ws=None) == 4 and _mm(M=40, K=63, ws=0x8000010) == 4
    assert _mm(M=40, K=63, ws=0x2000000) == 1                         # workspace over w
    assert _mm(M=0) == 0 and _mm(N=0) == 0


def test_matmul_workspace():
    sz = ctypes.c_size_t()
    f = bnd.load().dora_matmul_workspace_size

    def size(M, N, K, r, dtype, al=15):
        assert f(M, N, K, r, dtype, al, ctypes.byref(sz)) == 0
        return sz.value

    assert size(8192, 8192, 8192, 384, 0) == 0                  # aligned and enough tiles: nothing
    assert size(0, 8192, 8192, 384, 0) == 0
    # rows that are no multiple of 16 bytes, or operands that do not start on one, are copied
    assert size(4096, 4096, 4095, 0, 0) >= 2 * 4096 * 4096 * 2
    assert size(4096, 4096, 4096, 0, 0, al=13) >= 4096 * 4096 * 2
    assert size(4096, 4096, 4096, 0, 3) == 0
    assert f(4, 4, 4, 0, 4, 15, ctypes.byref(sz)) == 2
    assert f(4, 4, 4, 0, 0, 15, None) == 1 and f(-4, 4, 4, 0, 0, 15, ctypes.byref(sz)) == 1


def test_matmul_plans_cover_every_kernel():
    # (the shapes of the GPU tests' coverage list; see test_gpu_matmul.py)
    def plan(*a, **k):
        p = bnd.dora_matmul_plan_info(*a, **k)
        return p["tile_rows"], p["splits"] > 1, p["copies"]

    assert plan(8192, 8192, 8192, 384, "bf16") == (256, False, 0)
    assert plan(16, 28672, 8192, 0, "e4m3")[0] == 0 and plan(32, 64, 64, 0, "bf16")[0] == 0
    assert plan(33, 64, 64, 0, "bf16")[0] == 64
    assert plan(64, 8192, 8192, 0, "bf16")[1]
    assert plan(333, 1001, 777, 24, "f16") == (64, False, 3)
    assert plan(333, 1001, 777, 20, "f16")[2] == 15 and plan(333, 1001, 776, 24, "f16", aligned_operands=11)[2] == 4
    assert bnd.dora_matmul_plan_info(0, 8, 8, 0, "bf16")["tile_rows"] == -1
    f, info = bnd.load().dora_matmul_plan_info, (ctypes.c_int64 * 6)()
    assert f(64, 64, 64, 0, 0, 15, info, 6) == 0 and info[4] == info[5] == -1
    assert f(64, 64, 64, 0, 0, 15, None, 4) == 1 and f(64, 64, 64, 0, 9, 15, info, 4) == 2


def _mm_bwd(dy=0x1000000, u=0x2000000, x=0x3000000, w=0x4000000, dtype=0, M=4, N=32, K=64, col_scale=None, bias=None,
            act=0, du=None, dx=0x5000000, dw=0x6000000, dbias=0x7000000, dcol=0x7100000, ws=0x8000000,
            ws_bytes=1 << 24):
    return bnd.load().dora_matmul_backward(P(dy), P(u), P(x), P(w), dtype, M, N, K, P(col_scale), P(bias), act, P(du),
                                           P(dx), P(dw), P(dbias), P(dcol), P(ws), ws_bytes, None)


def test_matmul_backward_refusals():
    assert _mm_bwd(dtype=3) == 2
    assert _mm_bwd(M=-1) == 1 and _mm_bwd(N=1 << 22) == 1 and _mm_bwd(M=1 << 22) == 1
    assert _mm_bwd(act=9) == 1
    assert _mm_bwd(dy=None) == 1 and _mm_bwd(u=None) == 1 and _mm_bwd(x=None) == 1 and _mm_bwd(w=None) == 1
    assert _mm_bwd(dx=0x3000000) != 0 and _mm_bwd(dx=0x6000000) == 1
    assert _mm_bwd(dx=0x1000002) == 1
    assert _mm_bwd(dbias=0x7100000) == 1
    assert _mm_bwd(ws_bytes=16) == 4 and _mm_bwd(ws=None) == 4
    sz = ctypes.c_size_t()
    f = bnd.load().dora_matmul_backward_workspace_size
    assert f(4, 32, 64, 0, 32, ctypes.byref(sz)) == 1 and f(4, 32, 64, 3, 1, ctypes.byref(sz)) == 2
    assert f(4, 32, 64, 0, 15, None) == 1


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        bnd.dora_rms_norm(x, None, 1e-6)
    with pytest.raises(ValueError):
        bnd.dora_matmul(x, x)
    with pytest.raises(TypeError):
        bnd.dora_matmul(None, x)
    with pytest.raises(ValueError):
        bnd.dora_matmul_backward(x, x, x, x)
    with pytest.raises(TypeError):
        bnd.dora_matmul_workspace_size(4, 4, 4, 0, torch.int8)


def test_matmul_backward_refuses_a_bad_row_scale():
    def call(row_scale, du=None, ws=0x8000000):
        return bnd.load().dora_matmul_backward_rows(P(0x1000000), P(0x2000000), P(0x3000000), P(0x4000000), 0, 4, 32, 64,
                                                    P(row_scale), None, None, 0, P(du), P(0x5000000), P(0x6000000),
                                                    None, None, P(ws), 1 << 24, None)

    assert call(0x9000002) == 1
    assert call(0x5000000) == 1 and call(0x6000004) == 1 and call(0x7000000, du=0x7000000) == 1
    assert call(0x8000010) == 1                                 # in the workspace
    assert call(0x9000000, ws=None) == 4


def test_matmul_backward_takes_every_depth_that_the_product_takes():
    sz = ctypes.c_size_t()
    lib = bnd.load()
    for M, N, K in ((16, 8, 100000), (8, 100000, 16), (100000, 8, 16), (16, 8, (1 << 22) - 8)):
        assert lib.dora_matmul_workspace_size(M, N, K, 0, 0, 15, ctypes.byref(sz)) == 0
        assert lib.dora_matmul_backward_workspace_size(M, N, K, 0, 31, ctypes.byref(sz)) == 0, (M, N, K)
        assert _mm_bwd(M=M, N=N, K=K, x=0x10000000, w=0x30000000, dx=0x50000000, dw=0x70000000, ws=None) == 4
    assert lib.dora_matmul_backward_workspace_size(16, 8, 1 << 22, 0, 31, ctypes.byref(sz)) == 1
    assert lib.dora_matmul_backward_workspace_size(16, 1 << 22, 8, 0, 31, ctypes.byref(sz)) == 1
    assert lib.dora_matmul_backward_workspace_size(1 << 22, 16, 8, 0, 31, ctypes.byref(sz)) == 1


def test_which_blocks_few_rows_take():
    def few(M, N, K, dtype, r=0):
        return bnd.dora_matmul_plan_info(M, N, K, r, dtype)["few_rows"]

    assert few(1, 8192, 8192, "bf16") == few(8, 300, 64, "f32") == 8
    assert few(9, 8192, 8192, "bf16") == few(16, 28672, 8192, "e4m3") == 16
    # 17 to 32 rows: more than one round of 16 x 16, or a long depth of enough columns
    for M in (17, 32):
        for dtype in ("bf16", "f16", "f32", "e4m3"):
            assert few(M, 2064, 1024, dtype) == 32 and few(M, 2048, 1024, dtype) == 16
        assert few(M, 1001, 8189, "f16") == 32 and few(M, 1001, 8192, "bf16") == 32
        assert few(M, 1001, 4093, "f16") == 16 and few(M, 2048, 4096, "bf16") == 16
        assert few(M, 2048, 16384, "e4m3") == 32 and few(M, 2048, 8192, "e4m3") == 16
        assert few(M, 2048, 8192, "f32") == 16 and few(M, 256, 32765, "f16") == 16
    assert few(64, 256, 256, "f32") == 16 and few(64, 64, 64, "bf16") == -1


def test_rows_past_a_launch_are_refused():
    sz = ctypes.c_size_t()
    f = bnd.load().dora_matmul_workspace_size
    # a 64-row tile has 256 threads: 2^30 rows are 2^32 threads, more than a launch takes
    assert f(1 << 30, 4, 4, 0, 0, 15, ctypes.byref(sz)) == 1
    assert f((1 << 30) - 1, 4, 4, 0, 0, 15, ctypes.byref(sz)) == 0
    far = dict(x=0x1000000, w=0x2000000, col_scale=None, bias=None, y=0x10_0000_0000, ws=0x100_0000_0000)
    assert _mm(M=1 << 30, N=4, K=4, **far) == 1
    assert _mm(M=4, N=1 << 23, K=4) == 1 and _mm(M=1 << 17, N=64, K=1 << 17) == 1
