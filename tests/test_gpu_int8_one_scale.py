"""The backward's products with rows of one scale each, whose significands are in the other operand.

Tolerances. The other operand is du times a factor, rounded once, so it is off by half a step of itself as du is (fp16's
smallest step, 2^-24, counts up to twice: the factor is a half or more); the rows' own values are exact. In the 2-norm a
rounding of values that are spread evenly over a binade's logarithm is half a step times (1/3)^(1/2) (3 / (8 ln 2))^(1/2)
= 0.425 of it; the operand's and the result's are independent, 0.601 of half a step together, where rounding the rows too
makes 0.736.
"""

import ctypes

import numpy as np
import pytest
import torch

from block_helpers import EPS32, HALF, TINY, TORCH_DT, close, draw, host, rounded, vec
from dora_weight_norm_amd import binding as bnd
from oracle import block_oracle as B
from test_gpu_int8 import ACTS, off, values

pytestmark = pytest.mark.gpu


def rows_of(rng, shape, dtype, std=1.0, group=0):
    return bnd.Int8Rows(*bnd.dora_quantize_rows(draw(rng, shape, dtype, std), group=group), group)


def check(got, dy, u, x, w, c, bias, name, dtype, rows=None):
    M, N = dy.shape
    hdy, hu, hx, hw, hc, hb = host(dy), values(u), values(x), values(w), host(c), host(bias)
    du = B.matmul_backward(hdy, hu, hx, hw, hc, hb, name)[4]
    z = B.preactivation(hu, hc, hb)
    edz = np.abs(hdy) * (6 * EPS32 * np.abs(z) + (0 if name in ("none", "relu") else 16 * EPS32 * (1 + np.abs(z))))
    if name == "relu":
        edz = edz + np.abs(hdy) * (np.abs(z) <= 4 * EPS32 * (np.abs(z) + np.abs(hu) * 2 + 2))
    edz = edz + 2 * EPS32 * np.abs(hdy)
    C = np.abs(hc)[None, :]
    if rows is not None:
        du, C = du * host(rows)[:, None], C * np.abs(host(rows))[:, None]
    e32 = C * edz + 3 * EPS32 * np.abs(du)
    close(got[4], du, rounded(dtype, du, e32), "du")
    tol = rounded(dtype, du, e32) + TINY[dtype]
    adu = np.abs(du) + tol
    for i, out, a, n, what in ((0, lambda v, a: v @ a, hw, N, "dx"), (1, lambda v, a: v.T @ a, hx, M, "dw")):
        if got[i] is not None:
            ref, aa = out(du, a), np.abs(a)
            close(got[i], ref, rounded(dtype, ref, (n + 4) * EPS32 * out(adu, aa) + out(tol, aa)), what)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(8200, 384, 4112), (4100, 1024, 2064), (64, 128, 256), (333, 1001, 777), (17, 129, 77), (1, 1, 1),
                                   (1544, 2568, 264), (100, 1000, 8208), (2048, 2048, 64)])
def test_products_with_rows_of_one_scale(M, N, K, dtype):
    rng = np.random.default_rng(M + K)
    name = ACTS[(M + N + K) % 5]
    dy, u = draw(rng, (M, N), dtype), rows_of(rng, (M, N), dtype, group=64)
    x, w = rows_of(rng, (M, K), dtype), rows_of(rng, (N, K), dtype, K ** -0.5)
    c, bias = vec(rng, N, 0.2), vec(rng, N, 0.3, 0.0)
    got = bnd.dora_matmul_backward_int8(dy, u, x, w, col_scale=c, bias=bias, act=name)
    check(got, dy, u, x, w, c, bias, name, dtype)
    for v, k in ((x, "x"), (w, "w")):       # (one group of all columns is one scale too)
        if K <= 256:
            same = dict(x=x, w=w)
            same[k] = bnd.Int8Rows(v.q, v.scale.view(-1, 1), 256)
            again = bnd.dora_matmul_backward_int8(dy, u, same["x"], same["w"], col_scale=c, bias=bias, act=name)
            for a, b in zip(again, got):
                assert torch.equal(a, b)
    rows = vec(rng, M, 0.4)
    got = bnd.dora_matmul_backward_int8(dy, u, x, w, row_scale=rows, col_scale=c, bias=bias, act=name)
    check(got, dy, u, x, w, c, bias, name, dtype, rows)


# (read as they are held by tiles of 256 and of 128 rows, and brought back)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(4096, 1024, 4096), (1024, 2048, 1024), (600, 500, 1001)])
def test_two_roundings_and_not_three(M, N, K, dtype):
    rng = np.random.default_rng(5)
    dy, u = draw(rng, (M, N), dtype), draw(rng, (M, N), dtype)
    x, w = rows_of(rng, (M, K), dtype), rows_of(rng, (N, K), dtype, K ** -0.5)
    c, bias = vec(rng, N, 0.2), vec(rng, N, 0.3, 0.0)
    got = bnd.dora_matmul_backward_int8(dy, u, x, w, col_scale=c, bias=bias, act="silu")
    dx, dw = B.matmul_backward(host(dy), host(u), values(x), values(w), host(c), host(bias), "silu")[:2]
    for g, r in ((got[0], dx), (got[1], dw)):
        assert np.linalg.norm(host(g) - r) / np.linalg.norm(r) <= 0.65 * HALF[dtype]


@pytest.mark.parametrize("needs", [(1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("forms", [(0, 0), (0, None), (None, 0), (0, 32), (32, 0)])
@pytest.mark.parametrize("M,N,K", [(70, 136, 200), (33, 77, 129)])
def test_outputs_du_and_workspace(M, N, K, forms, needs):
    """With du, without, in the place of dy; workspaces of just the queried size, between bytes that stay."""
    rng = np.random.default_rng(6)
    dy, u = draw(rng, (M, N), "bf16"), draw(rng, (M, N), "bf16")

    def held(shape, group):
        return draw(rng, shape, "bf16") if group is None else rows_of(rng, shape, "bf16", group=group)

    x, w = held((M, K), forms[0]), held((N, K), forms[1])
    ndx, ndw = map(bool, needs)
    want = bnd.dora_matmul_backward_int8(dy, u, x, w, act="silu", need_dx=ndx, need_dw=ndw)
    args = []
    for v, need in ((x, ndw), (w, ndx)):
        a8 = bnd._Int8RowsArg(v.q.data_ptr(), v.scale.data_ptr(), v.group) if need and isinstance(v, bnd.Int8Rows) else None
        args.append((None if a8 or not need else v.data_ptr(), None if a8 is None else ctypes.byref(a8), a8))
    scales = [0 if f is None else (-(-K // f) if f else 1) for f in forms]
    for du_at in ("none", "own", "dy"):
        y, du = dy.clone(), torch.full_like(dy, 9)
        pdu = {"none": None, "own": du.data_ptr(), "dy": y.data_ptr()}[du_at]
        outputs = (bnd.GRAD_DX * ndx + bnd.GRAD_DW * ndw + bnd.GRAD_SUMS + bnd.GRAD_DU * (du_at != "none") + bnd.GRAD_ALIGNED)
        need = bnd._size_of("dora_matmul_backward_int8_scales_workspace_size", M, N, K, 0, outputs,
                            scales[0] * ndw, scales[1] * ndx)
        ws = torch.full((need + 512,), 0x5a, device="cuda", dtype=torch.uint8)
        outs = [torch.empty_like(v) if v is not None else None for v in want[:4]]
        bnd._call("dora_matmul_backward_int8", y.data_ptr(), u.data_ptr(), None, args[0][0], args[0][1], args[1][0],
                  args[1][1], 0, M, N, K, None, None, None, 4, pdu, *(bnd._addr(v) for v in outs), ws.data_ptr() + 256, need,
                  torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        for g, r in zip(outs, want):
            assert r is None or torch.equal(g, r), du_at
        if du_at != "none":
            assert torch.equal(du if du_at == "own" else y, want[4])
        assert (ws[:256] == 0x5a).all() and (ws[256 + need:] == 0x5a).all()


@pytest.mark.parametrize("dtype,scales", [("bf16", [2.0 ** -100, 2.0 ** -60, 1.99 * 2.0 ** -20, 1, 0.75 * 2.0 ** 60, 2.0 ** 90]),
                                          ("f16", [2.0 ** -24, 1.5 * 2.0 ** -20, 2.0 ** -14, 0.7, 255.9, 257.0, 511.0, 515.78])])
@pytest.mark.parametrize("M,N,K", [(2048, 1024, 2048), (72, 40, 48)])
def test_scales_of_every_size(M, N, K, dtype, scales):
    """One row of x at a time meets a gradient: dw is its values times that, each rounded once to the type."""
    rng = np.random.default_rng(7)
    q = torch.from_numpy(rng.integers(-127, 128, (M, K)).astype(np.int8)).cuda()
    q[:, :3] = torch.tensor([-128, 127, 0], dtype=torch.int8)
    s = torch.tensor(np.resize(scales, M).astype(np.float32)).cuda()
    for m in range(len(scales)):
        dy = torch.zeros(M, N, device="cuda", dtype=TORCH_DT[dtype])
        dy[m] = 2.0 ** -2
        dw = bnd.dora_matmul_backward_int8(dy, dy, bnd.Int8Rows(q, s), None, need_dx=False)[1]
        ref = host(q)[m] * float(s[m]) / 4
        # (the factor's rounding and the result's)
        tol = HALF[dtype] * 2.01 * np.abs(ref) + TINY[dtype]
        close(dw, np.broadcast_to(ref, (N, K)), np.broadcast_to(tol, (N, K)), f"dw {scales[m]}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(2048, 1024, 2048), (72, 40, 48)])
def test_scales_that_are_no_numbers_and_zeros(M, N, K, dtype):
    rng = np.random.default_rng(8)
    dy = draw(rng, (M, N), dtype)
    x, w = rows_of(rng, (M, K), dtype), rows_of(rng, (N, K), dtype)
    for bad in (float("nan"), float("inf")):
        xs, q = x.scale.clone(), x.q.clone()
        xs[M - 1], q[M - 1] = bad, 0
        dw = bnd.dora_matmul_backward_int8(dy, dy, bnd.Int8Rows(q, xs), None, need_dx=False)[1]
        assert torch.isnan(dw).all()
        ws, q = w.scale.clone(), w.q.clone()
        ws[3], q[3] = bad, 0
        assert torch.isnan(bnd.dora_matmul_backward_int8(dy, dy, None, bnd.Int8Rows(q, ws), need_dw=False)[0]).all()
    zero = w.scale.clone()
    zero[3] = 0                                  # a row that a scale of 0 makes 0
    plain = w.q.clone()
    plain[3] = 0
    a = bnd.dora_matmul_backward_int8(dy, dy, None, bnd.Int8Rows(w.q, zero), need_dw=False)[0]
    b = bnd.dora_matmul_backward_int8(dy, dy, None, bnd.Int8Rows(plain, w.scale), need_dw=False)[0]
    assert torch.equal(a, b)


def test_rows_of_one_scale_off_the_grid_on_a_stream_and_in_a_graph():
    rng = np.random.default_rng(9)
    M, N, K = 300, 264, 528
    dy, u = draw(rng, (M, N), "bf16"), draw(rng, (M, N), "bf16")
    x, w = rows_of(rng, (M, K), "bf16"), rows_of(rng, (N, K), "bf16")
    c, bias = vec(rng, N, 0.2), vec(rng, N, 0.3, 0.0)
    moved = [bnd.Int8Rows(off(v.q), off(v.scale)) for v in (x, w)]
    got = bnd.dora_matmul_backward_int8(off(dy), off(u), *moved, col_scale=off(c), bias=off(bias), act="gelu")
    check(got, dy, u, x, w, c, bias, "gelu", "bf16")

    def step(**kw):
        return bnd.dora_matmul_backward_int8(dy, u, x, w, col_scale=c, bias=bias, act="gelu", **kw)

    want = step()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    side = step(stream=st)
    st.synchronize()
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        inside = step()
    for _ in range(3):
        for v in inside:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, d in zip(inside, want, side):
            assert torch.equal(a, b) and torch.equal(d, b)
        eager = step()
        torch.cuda.synchronize()
        for a, b in zip(eager, want):
            assert torch.equal(a, b)


# Rows in groups beside a dy that is an operand as it is: brought back, and read by tiles of 128 (in parts) and 256 rows.
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,reads", [(8200, 384, 4112, "int8_rows"), (4096, 2048, 4096, "int8_rows"), (600, 504, 1000, "copy"),
                                         (64, 1000, 128, "copy")])
def test_without_an_activation_dy_is_the_operand(M, N, K, reads, dtype):
    assert bnd.dora_matmul_backward_int8_plan_info(M, N, K, dtype, x_scales=9, w_scales=0)["dw"]["reads"] == reads
    rng = np.random.default_rng(10)
    dy, u, w = draw(rng, (M, N), dtype), rows_of(rng, (M, N), dtype, group=32), draw(rng, (N, K), dtype, K ** -0.5)
    x, c, bias = rows_of(rng, (M, K), dtype, group=64), vec(rng, N, 0.2), vec(rng, N, 0.3, 0.0)
    got = bnd.dora_matmul_backward_int8(dy, u, x, w, col_scale=c, bias=bias)
    dw = (host(dy) * host(c)[None, :]).T @ values(x)
    assert np.linalg.norm(host(got[1]) - dw) / np.linalg.norm(dw) <= 0.65 * HALF[dtype]
    size = np.abs(host(dy) * host(c)[None, :]).T @ np.abs(values(x))
    close(got[1], dw, rounded(dtype, dw, (HALF[dtype] * 1.01 + (M + 4) * EPS32) * size + TINY[dtype] * np.abs(host(c)).max()
                              * np.abs(host(dy)).sum(0)[:, None]), "dw")
    # off the boundary, and in du's place, du is the operand
    for other in (off(dy), dy):
        again = bnd.dora_matmul_backward_int8(other, u, x, w, col_scale=c, bias=bias)
        assert torch.equal(again[0], got[0]) and torch.equal(again[4], got[4])
        close(again[1], dw, rounded(dtype, dw, (HALF[dtype] * 2.02 + (M + 4) * EPS32) * size + 3 * TINY[dtype]
                                    * (np.abs(host(dy)).sum(0)[:, None] + np.abs(values(x)).sum(0)[None, :])), "dw")
    y, x8 = dy.clone(), bnd._Int8RowsArg(x.q.data_ptr(), x.scale.data_ptr(), 64)
    need = bnd._size_of("dora_matmul_backward_int8_scales_workspace_size", M, N, K, bnd._dtype_code(dtype),
                        bnd.GRAD_DW + bnd.GRAD_DU + bnd.GRAD_ALIGNED, -(-K // 64), 0)
    ws, into = torch.empty(need + 16, device="cuda", dtype=torch.uint8), torch.empty_like(got[1])
    back = host(bnd.dora_dequantize_rows(*u, dtype=torch.float32))
    uu = torch.from_numpy(back).cuda().to(dy.dtype)
    bnd._call("dora_matmul_backward_int8", y.data_ptr(), uu.data_ptr(), None, None, ctypes.byref(x8), None, None,
              bnd._dtype_code(dtype), M, N, K, None, c.data_ptr(), None, 0, y.data_ptr(), None, into.data_ptr(), None, None,
              ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(y, got[4])
    close(into, dw, rounded(dtype, dw, (HALF[dtype] * 2.02 + (M + 4) * EPS32) * size + 3 * TINY[dtype]
                            * (np.abs(host(dy)).sum(0)[:, None] + np.abs(values(x)).sum(0)[None, :])), "dw")


@pytest.mark.parametrize("kw", [dict(act="relu"), dict(rows=True), dict()])
def test_du_is_the_operand_elsewhere(kw):
    """With an activation, a row scale, or no column scale (du is dy then)."""
    rng = np.random.default_rng(11)
    M, N, K = 300, 264, 520
    dy, u, w = draw(rng, (M, N), "bf16"), draw(rng, (M, N), "bf16"), draw(rng, (N, K), "bf16")
    x = rows_of(rng, (M, K), "bf16", group=64)
    c = vec(rng, N, 0.2) if kw else None
    rows = vec(rng, M, 0.4) if "rows" in kw else None
    got = bnd.dora_matmul_backward_int8(dy, u, x, w, col_scale=c, act=kw.get("act", "none"), row_scale=rows)
    if c is None:
        assert torch.equal(got[4], dy)
    du, xv = host(got[4]), values(x)
    ref, size = du.T @ xv, np.abs(du).T @ np.abs(xv)
    close(got[1], ref, rounded("bf16", ref, (HALF["bf16"] * 1.01 + (M + 4) * EPS32) * size), "dw")
