"""Rows in 8-bit integers on the GPU: packing, the integer product, and the backward that reads packed operands, against
the fp64 reference.

Tolerances. Packing is exact: the scale is one fp32 division and a value the whole number nearest to its quotient.
A product's integer sum is exact; converted in at most 48 parts (eight waves by two halves, or 32 parts of a depth)
that are each rounded once, scaled by two roundings and added, it is off by 56 2^-24 of the sum of its products'
sizes. A pair of depth r is added in fp32 onto it. Epilogue and outputs as in test_gpu_matmul.py, whose backward
bounds hold with the operands' own rounding to the storage type added.
"""

import numpy as np
import pytest
import torch

from block_helpers import EPS32, HALF, TINY, TORCH_DT, close, draw, host, rounded, vec
from dora_weight_norm_amd import binding as bnd
from oracle import block_oracle as B
from oracle import int8_oracle as Q

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
GROUPS = [0, 32, 64, 128, 256]
ROWS = [(1, 1), (1, 8), (3, 31), (2, 32), (5, 33), (4, 127), (7, 128), (1, 256), (3, 257), (64, 512), (600, 1000),
        (513, 2049), (1, 8192), (33, 8200), (2, 16384), (2, 16385), (2, 40003), (530, 4096), (2100, 4096), (9000, 1000),
        (0, 64)]


def pack(rng, shape, std=1.0):
    """(int8 tensor, scale) of random rows, packed by the reference."""
    q, s = Q.quantize_rows((rng.standard_normal(shape) * std).astype(np.float32))
    return torch.from_numpy(q.astype(np.int8)).cuda(), torch.from_numpy(s.astype(np.float32)).cuda()


def off(t):
    """The same values one element into a buffer."""
    b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
    b.copy_(t)
    return b


# ---------------------------------------------------------------- packing

@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,d", ROWS)
def test_packing_is_exact(T, d, dtype):
    rng = np.random.default_rng(T * 31 + d)
    x = draw(rng, (T, d), dtype)
    if T:
        x[:, rng.integers(0, d)] *= 20
        x[T // 2, : d // 2] = 0
    for group in GROUPS:
        q, s = bnd.dora_quantize_rows(x, group=group)
        if T == 0:
            assert q.shape == (0, d) and s.shape == ((0, -(-d // group)) if group else (0,))
            continue
        rq, rs = Q.quantize_rows(host(x), group)
        assert np.array_equal(s.cpu().numpy(), rs), group
        assert np.array_equal(host(q), rq), (group, np.abs(host(q) - rq).max())
        for out in ("bf16", "f16", "f32"):
            back = bnd.dora_dequantize_rows(q, s, group=group, dtype=TORCH_DT[out])
            ref = q.float() * torch.from_numpy(np.repeat(rs.reshape(T, -1), group or d, 1)[:, :d]).cuda()
            assert torch.equal(back, ref.to(TORCH_DT[out])), (group, out)


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_ties_go_to_the_even_step(dtype, group):
    """Values on and beside the borders of two steps, under scales that make the borders ties or not."""
    rng = np.random.default_rng(3)
    T, d = 300, 1024
    x = (rng.integers(-127, 127, (T, d)) + 0.5) * rng.choice([1, 2.0 ** -7, 1 + 2.0 ** -6], (T, 1))
    x[:, ::32] = 127 * rng.choice([1, 2, 1 + 2.0 ** -7, 0.5], (T, 32))
    x = torch.from_numpy(x.astype(np.float32)).cuda().to(TORCH_DT[dtype])
    q, s = bnd.dora_quantize_rows(x, group=group)
    rq, rs = Q.quantize_rows(host(x), group)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(host(q), rq)
    halves = np.abs(host(x) / Q.dequantize_rows(np.ones((T, d)), rs, group) % 1)
    assert (halves == 0.5).sum() > 1000          # (the inputs do what they are for)


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("T,d", [(6, 512), (600, 300), (6, 20000)])
def test_packing_special_values(T, d, group):
    rng = np.random.default_rng(4)
    x = draw(rng, (T, d), "f32")
    x[0] = 0
    x[1, 3], x[2, 5], x[3, 7] = float("nan"), float("inf"), float("-inf")
    x[4] *= 1e-35                                # scales below the least
    x[5] *= 1e37
    q, s = bnd.dora_quantize_rows(x, group=group)
    v = host(bnd.dora_dequantize_rows(q, s, group=group, dtype=torch.float32))
    g = group or d
    assert (host(s)[0] == 1).all() and not host(q)[0].any()
    for row in (1, 2, 3):
        assert np.isnan(v[row, :g]).all() and np.isfinite(v[row, g:]).all() and not host(q)[row, :g].any()
    assert (host(s)[4] == 2.0 ** -100).all()
    rq, rs = Q.quantize_rows(host(x)[4:], group)
    assert np.array_equal(s[4:].cpu().numpy(), rs) and np.array_equal(host(q)[4:], rq)


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("T,d", [(5, 264), (40, 777), (3, 9001)])
def test_packing_unaligned_streams_and_repeats(T, d, group):
    rng = np.random.default_rng(5)
    x = draw(rng, (T, d), "bf16")
    q, s = bnd.dora_quantize_rows(x, group=group)
    q2, s2 = bnd.dora_quantize_rows(off(x), group=group, q=off(q), scale=off(s))
    assert torch.equal(q, q2) and torch.equal(s, s2)
    v = bnd.dora_dequantize_rows(q, s, group=group)
    assert torch.equal(v, bnd.dora_dequantize_rows(off(q), off(s), group=group, out=off(v)))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    q3, s3 = bnd.dora_quantize_rows(x, group=group, stream=st)
    v3 = bnd.dora_dequantize_rows(q3, s3, group=group, stream=st)
    st.synchronize()
    assert torch.equal(q, q3) and torch.equal(s, s3) and torch.equal(v, v3)


def test_packing_offsets_past_32_bits():
    T, d, n = 530001, 8200, 20
    rng = np.random.default_rng(6)
    x = torch.zeros(T, d, device="cuda", dtype=torch.bfloat16)
    x[-n:] = draw(rng, (n, d), "bf16")
    for group in (0, 128):
        q, s = bnd.dora_quantize_rows(x, group=group)
        rq, rs = Q.quantize_rows(host(x[-n:]), group)
        assert np.array_equal(s[-n:].cpu().numpy(), rs) and np.array_equal(host(q[-n:]), rq)
        assert not q[:-n].any() and (s[:-n] == 1).all()
        v = bnd.dora_dequantize_rows(q, s, group=group)
        assert torch.equal(v[-n:], bnd.dora_dequantize_rows(q[-n:].clone(), s[-n:].clone(), group=group))
        del v, q, s


# ---------------------------------------------------------------- the integer product

def operands(M, N, K, r, out, seed):
    rng = np.random.default_rng(seed)
    x, xs = pack(rng, (M, max(K, 1)))
    w, ws = pack(rng, (N, max(K, 1)), max(K, 1) ** -0.5)
    o = {"x": x[:, :K].contiguous(), "w": w[:, :K].contiguous(), "row_scale": xs, "w_scale": ws,
         "col_scale": vec(rng, N, 0.2), "bias": vec(rng, N, 0.3, 0.0)}
    if r:
        o.update(t=draw(rng, (M, r), out), b=draw(rng, (N, r), out, 0.1), s=0.5)
    return o, rng


def product(o):
    """(u, bound of its fp32 error) in fp64."""
    x, w = host(o["x"]), host(o["w"])
    sc = host(o["row_scale"])[:, None] * host(o["w_scale"])[None, :]
    u, size = x @ w.T * sc, np.abs(x) @ np.abs(w).T * np.abs(sc)
    r = 0
    if o.get("t") is not None:
        t, b = host(o["t"]), host(o["b"])
        r = t.shape[1]
        u = u + o["s"] * (t @ b.T)
        pair = abs(o["s"]) * (np.abs(t) @ np.abs(b).T)
        return u, (56 + 4 + r) * EPS32 * size + (56 + r + 4) * EPS32 * pair
    return u, 56 * EPS32 * size


def check(o, rng, out, name, with_residual, save):
    M, N = o["x"].shape[0], o["w"].shape[0]
    res = draw(rng, (M, N), out) if with_residual else None
    u, eu = product(o)
    c, bias = host(o.get("col_scale")), host(o.get("bias"))
    z = B.preactivation(u, c, bias)
    y = B.act(z, name)
    C = 1.0 if c is None else np.abs(c)[None, :]
    ey = 1.13 * (C * eu + 2 * EPS32 * (C * np.abs(u) + np.abs(z)))
    ey = ey + (0 if name == "none" else 8 * EPS32 * np.abs(z) * (1 + np.abs(z)))
    if res is not None:
        y = y + host(res)
        ey = ey + EPS32 * (np.abs(y) + np.abs(host(res)))
    gy, gu = bnd.dora_matmul_int8(**o, act=name, residual=res, save=save, out_dtype=TORCH_DT[out])
    assert gy.dtype == TORCH_DT[out] and (gu is not None) == save
    if save:
        close(gu, u, rounded(out, u, eu + 2 * EPS32 * np.abs(u)), "u")
    close(gy, y, rounded(out, y, ey), "y")


SHAPES = [(1, 1, 1, 0), (1, 257, 512, 0), (1, 512, 4096, 64), (2, 40, 64, 3), (5, 96, 2048, 16), (16, 130, 520, 0),
          (17, 300, 777, 24), (33, 64, 8192, 0), (64, 256, 256, 8), (100, 1000, 40, 0), (128, 128, 64, 64),
          (333, 1001, 777, 24), (256, 255, 0, 16), (300, 520, 1032, 130), (1000, 700, 130, 64), (513, 1544, 136, 0),
          (2050, 6410, 72, 8), (1, 3, 0, 0), (1, 100, 5000, 40), (7, 33, 1023, 5), (15, 31, 16, 700), (2, 64, 20001, 0),
          (32, 4200, 1024, 8), (250, 255, 520, 0), (49, 17, 8200, 16)]


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,r", SHAPES)
def test_int8_product(M, N, K, r, out):
    o, rng = operands(M, N, K, 0 if out == "f32" else r, out, M + 31 * N + 7 * K)
    check(o, rng, out, ACTS[(M + N + K) % 5], (M + K) % 2 == 0, N % 2 == 0)


# One shape for each kernel and what may come with it: (M, N, K, r, tile rows, split depth).
COVER = [(4100, 4104, 528, 0, 256, False), (4100, 4104, 528, 40, 256, False), (1030, 4104, 4112, 0, 128, None),
         (1030, 4104, 1040, 24, 128, None), (70, 520, 8208, 16, 64, True), (70, 520, 8208, 0, 64, True),
         (300, 520, 528, 16, 64, False), (16, 200, 16400, 16, 0, True), (70, 4104, 256, 1024, 64, None)]


@pytest.mark.parametrize("M,N,K,r,rows,split,out", [(*c, t) for c in COVER for t in ("bf16", "f16", "f32")
                                                     if t != "f32" or c[3] == 0])
def test_every_int8_kernel(M, N, K, r, rows, split, out):
    plan = bnd.dora_matmul_int8_plan_info(M, N, K, r)
    assert plan["tile_rows"] == rows and split in (None, plan["splits"] > 1), plan
    o, rng = operands(M, N, K, r, out, M + K)
    check(o, rng, out, ACTS[1 + K // 16 % 4], K % 32 == 16, True)


@pytest.mark.parametrize("M,N,K", [(1, 40, 700), (16, 130, 1000), (32, 4200, 640), (40, 70, 1023), (70, 520, 8208),
                                   (300, 520, 528), (1030, 4104, 512), (4100, 4104, 272)])
def test_integer_sums_are_exact(M, N, K):
    """Scales of 1, fp32 outputs and sums below 2^24: the whole number itself."""
    rng = np.random.default_rng(7)
    lim = int(min(127, (2 ** 24 / K) ** 0.5))
    x, w = (torch.from_numpy(rng.integers(-lim, lim + 1, s).astype(np.int8)).cuda() for s in ((M, K), (N, K)))
    one = torch.ones(max(M, N), device="cuda")
    y, _ = bnd.dora_matmul_int8(x, w, one[:M], one[:N], out_dtype=torch.float32)
    assert torch.equal(y.double(), x.double() @ w.double().t())


@pytest.mark.parametrize("M", [1, 40, 300])
def test_the_longest_depth_of_the_largest_values(M):
    K, N = 131071, 64
    x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    one = torch.ones(max(M, N), device="cuda")
    y, _ = bnd.dora_matmul_int8(x, w, one[:M], one[:N], out_dtype=torch.float32)
    # (parts are rounded to fp32 and added)
    want = np.full(N, 128.0 * 128 * K)
    want[1] = -128.0 * 127 * K
    close(y, np.broadcast_to(want, (M, N)), 56 * EPS32 * np.abs(want), "y")


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("shape", [(40, 136, 192, 16), (3, 64, 4096, 0), (260, 400, 64, 8)])
def test_int8_activations(shape, name):
    o, rng = operands(*shape, "f16", 3)
    o["bias"] = vec(rng, shape[1], 4.0, 0.0)     # far into both tails
    check(o, rng, "f16", name, True, True)


@pytest.mark.parametrize("M", [3, 40, 300, 1030])
def test_scales_of_the_pair(M):
    """s of 0 leaves the pair unread (NaN in it stays out); s far from 1 and negative."""
    N, K, r = 264, 528, 24
    o, rng = operands(M, N, K, r, "bf16", 8)
    plain = {k: v for k, v in o.items() if k not in ("t", "b", "s")}
    want, _ = bnd.dora_matmul_int8(**plain)
    t = torch.full_like(o["t"], float("nan"))
    got, _ = bnd.dora_matmul_int8(**{**o, "t": t, "s": 0.0})
    assert torch.equal(got, want)
    for s in (-0.5, 2.0 ** -64, -2.0 ** 64, 1e-3, 37.0):
        o["s"] = s
        check(o, rng, "bf16", "none", False, True)


@pytest.mark.parametrize("M,r", [(1, 0), (4, 16), (40, 0), (40, 16), (300, 16), (300, 0)])
def test_int8_in_place_residual_unaligned_operands_and_repeats(M, r):
    N, K = 136, 272
    o, rng = operands(M, N, K, r, "bf16", 6)
    res = draw(rng, (M, N), "bf16")
    want, _ = bnd.dora_matmul_int8(**o, residual=res)
    again, _ = bnd.dora_matmul_int8(**o, residual=res)
    assert torch.equal(want, again)
    into = res.clone()
    bnd.dora_matmul_int8(**o, residual=into, y=into)
    assert torch.equal(into, want)
    moved = {k: (off(v) if k != "s" else v) for k, v in o.items()}
    got, _ = bnd.dora_matmul_int8(**moved, residual=off(res), y=off(res))
    assert torch.equal(got, want)


@pytest.mark.parametrize("r", [0, 16])
@pytest.mark.parametrize("M", [5, 70, 300])
def test_rows_with_a_nan_scale_stay_in_their_rows(M, r):
    o, _ = operands(M, 300, 528, r, "bf16", 7)
    clean, _ = bnd.dora_matmul_int8(**o)
    o["row_scale"][3] = float("nan")
    o["w_scale"][299] = float("inf")
    y, _ = bnd.dora_matmul_int8(**o)
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[:, 299]).any()
    keep = [i for i in range(M) if i != 3]
    assert torch.equal(y[keep, :299], clean[keep, :299])


def test_empty_int8_products():
    z = torch.empty(0, 64, device="cuda", dtype=torch.int8)
    w, one = torch.ones(8, 64, device="cuda", dtype=torch.int8), torch.ones(8, device="cuda")
    y, _ = bnd.dora_matmul_int8(z, w, one[:0], one)
    assert y.shape == (0, 8)
    y, _ = bnd.dora_matmul_int8(w[:3, :0].contiguous(), w[:, :0].contiguous(), one[:3], one, bias=2 * one)
    assert (y == 2).all()
    t = torch.ones(3, 4, device="cuda", dtype=torch.bfloat16)
    b = torch.ones(8, 4, device="cuda", dtype=torch.bfloat16)
    y, _ = bnd.dora_matmul_int8(w[:3, :0].contiguous(), w[:, :0].contiguous(), one[:3], one, t=t, b=b, s=0.5)
    assert (y == 2).all()


def test_int8_refusals_of_the_binding():
    i8, dev = torch.int8, "cuda"
    x, w = torch.zeros(4, 64, device=dev, dtype=i8), torch.zeros(8, 64, device=dev, dtype=i8)
    xs, ws = torch.ones(4, device=dev), torch.ones(8, device=dev)
    t, b = (torch.zeros(n, 2, device=dev, dtype=torch.bfloat16) for n in (4, 8))
    bad = [dict(w=w[:, :32]), dict(w=w.float()), dict(w=w.t()), dict(x=x.to(torch.uint8)), dict(row_scale=None),
           dict(w_scale=xs), dict(row_scale=xs.half()), dict(t=t), dict(t=t, b=b[:7]), dict(t=t.half(), b=b.half()),
           dict(t=t.float(), b=b.float(), out_dtype=torch.float32), dict(out_dtype=i8), dict(bias=xs), dict(act="tanh"),
           dict(residual=x), dict(y=x)]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            bnd.dora_matmul_int8(**{**dict(x=x, w=w, row_scale=xs, w_scale=ws), **kw})
    with pytest.raises(bnd.DoraError):
        bnd.dora_matmul_int8(x, w, xs, ws, t=t, b=b, s=1e-30)
    with pytest.raises(bnd.DoraError):
        bnd.dora_matmul_int8(x, w, xs, ws, s=float("inf"))
    with pytest.raises(ValueError):
        bnd.dora_matmul_int8(torch.zeros(40, 15, device=dev, dtype=i8), w[:, :15].contiguous(), torch.ones(40, device=dev),
                             ws, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    for bad in (dict(group=48), dict(q=x.float()), dict(scale=ws)):
        with pytest.raises((ValueError, TypeError)):
            bnd.dora_quantize_rows(t, **bad)
    with pytest.raises(TypeError):
        bnd.dora_quantize_rows(x)
    with pytest.raises(ValueError):
        bnd.dora_dequantize_rows(x, xs, group=32)
    with pytest.raises(TypeError):
        bnd.dora_dequantize_rows(x, xs, dtype=torch.float64)
    f = torch.zeros(4, 8, device=dev)
    rows = bnd.Int8Rows(torch.zeros(4, 8, device=dev, dtype=i8), xs)
    for u in (rows._replace(group=32), rows._replace(scale=ws), rows._replace(q=x), None, x):
        with pytest.raises((ValueError, TypeError)):
            bnd.dora_matmul_backward_int8(f, u, None, None, need_dx=False, need_dw=False)
    with pytest.raises(ValueError):
        bnd.dora_matmul_backward_int8(f, rows, None, f)


def test_int8_offsets_past_32_bits():
    """Rows of x and y far past 2^32 bytes in."""
    M, N, K = 524800, 4104, 4112
    rng = np.random.default_rng(9)
    w, ws = pack(rng, (N, K), K ** -0.5)
    x = torch.zeros(M, K, device="cuda", dtype=torch.int8)
    xs = torch.ones(M, device="cuda")
    n = 24
    tail, ts = pack(rng, (n, K))
    x[-n:], xs[-n:] = tail, ts
    y, _ = bnd.dora_matmul_int8(x, w, xs, ws)
    u, eu = product({"x": tail, "w": w, "row_scale": ts, "w_scale": ws})
    close(y[-n:], u, rounded("bf16", u, eu + 2 * EPS32 * np.abs(u)), "y")
    assert not y[:-n].any()


# ---------------------------------------------------------------- the backward

BWD = [(4100, 264, 4104), (264, 4104, 4112), (1, 1, 1), (3, 40, 64), (17, 129, 77), (64, 256, 256), (100, 264, 520),
       (333, 1001, 777), (600, 72, 1288), (1, 512, 640), (300, 2048, 64), (2000, 136, 128), (1544, 2568, 264)]


def backward_case(M, N, K, dtype, seed, gu, gx, gw):
    """(rng, dy, u, x, w, col_scale, bias) with u, x, w as Int8Rows of their groups (None: in the storage type)."""
    rng = np.random.default_rng(seed)

    def held(shape, std, group):
        v = draw(rng, shape, dtype, std)
        return v if group is None else bnd.Int8Rows(*bnd.dora_quantize_rows(v, group=group), group)

    return (rng, draw(rng, (M, N), dtype), held((M, N), 1.0, gu), held((M, K), 1.0, gx), held((N, K), K ** -0.5, gw),
            vec(rng, N, 0.2), vec(rng, N, 0.3, 0.0))


def values(v):
    return Q.dequantize_rows(host(v.q), host(v.scale), v.group) if isinstance(v, bnd.Int8Rows) else host(v)


def check_backward(got, dy, u, x, w, c, bias, name, dtype, rows=None):
    M, N = dy.shape
    H = [values(v) for v in (dy, u, x, w)] + [host(c), host(bias)]
    _, _, db, dc, du = B.matmul_backward(*H, name)
    z = B.preactivation(H[1], H[4], H[5])
    # (u's value itself is rounded to fp32; a relu's z beside 0 may change sides, where its slope is any of 0 to 1)
    edz = np.abs(H[0]) * (6 * EPS32 * np.abs(z) + (0 if name in ("none", "relu") else 16 * EPS32 * (1 + np.abs(z))))
    if name == "relu":
        edz = edz + np.abs(H[0]) * (np.abs(z) <= 4 * EPS32 * (np.abs(z) + np.abs(H[1]) * 2 + 2))
    edz = edz + 2 * EPS32 * np.abs(H[0])
    C = np.abs(H[4])[None, :] * (1.0 if rows is None else np.abs(host(rows))[:, None])
    if rows is not None:
        du = du * host(rows)[:, None]
    tol = rounded(dtype, du, C * edz + 2 * EPS32 * np.abs(du))
    close(got[4], du, tol, "du")

    def op(v, ref):   # error of an operand as the products take it
        return rounded(dtype, ref, EPS32 * np.abs(ref)) if isinstance(v, bnd.Int8Rows) else np.zeros_like(ref)

    adu = np.abs(du) + tol
    if got[0] is not None:
        dx, a = du @ H[3], np.abs(H[3])
        close(got[0], dx, rounded(dtype, dx, (N + 4) * EPS32 * (adu @ a) + tol @ a + adu @ op(w, H[3])), "dx")
    if got[1] is not None:
        dw, a = du.T @ H[2], np.abs(H[2])
        close(got[1], dw, rounded(dtype, dw, (M + 4) * EPS32 * (adu.T @ a) + tol.T @ a + adu.T @ op(x, H[2])), "dw")
    dz = np.abs(H[0] * B.slope(z, name))
    if got[2] is not None:
        close(got[2], db, (M + 4) * EPS32 * dz.sum(0) + edz.sum(0), "dbias")
    if got[3] is not None:
        close(got[3], dc, (M + 8) * EPS32 * (dz * np.abs(H[1])).sum(0) + (edz * np.abs(H[1])).sum(0), "dcol_scale")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", BWD)
def test_int8_backward(M, N, K, dtype):
    name = ACTS[(M + N + K) % 5]
    i = M + N + K
    gu, gx, gw = GROUPS[i % 5], GROUPS[(i + 2) % 5], (0 if i % 2 else None)
    rng, dy, u, x, w, c, bias = backward_case(M, N, K, dtype, M * 5 + N, gu, gx, gw)
    got = bnd.dora_matmul_backward_int8(dy, u, x, w, col_scale=c, bias=bias, act=name)
    check_backward(got, dy, u, x, w, c, bias, name, dtype)
    again = bnd.dora_matmul_backward_int8(dy, u, x, w, col_scale=c, bias=bias, act=name)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("forms", [(None, 0, 0), (0, None, 0), (64, 128, None), (None, None, 128), (256, 32, 64),
                                   (None, 64, None), (128, None, None), (None, None, None)])
@pytest.mark.parametrize("M,N,K", [(70, 136, 200), (33, 77, 129)])
def test_int8_backward_forms(M, N, K, forms, dtype):
    rng, dy, u, x, w, c, bias = backward_case(M, N, K, dtype, 3, *forms)
    got = bnd.dora_matmul_backward_int8(dy, u, x, w, col_scale=c, bias=bias, act="silu")
    check_backward(got, dy, u, x, w, c, bias, "silu", dtype)
    if forms == (None, None, None):
        for a, b in zip(got, bnd.dora_matmul_backward(dy, u, x, w, col_scale=c, bias=bias, act="silu")):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", ACTS)
def test_int8_backward_activations(name):
    rng, dy, u, x, w, c, bias = backward_case(60, 72, 40, "f32", 11, 32, 0, 0)
    got = bnd.dora_matmul_backward_int8(dy, u, x, w, col_scale=c, bias=bias, act=name)
    check_backward(got, dy, u, x, w, c, bias, name, "f32")


@pytest.mark.parametrize("needs", [(1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (1, 1, 0, 1)])
def test_int8_backward_of_some_outputs(needs):
    rng, dy, u, x, w, c, bias = backward_case(70, 88, 96, "bf16", 12, 64, 32, 0)
    full = bnd.dora_matmul_backward_int8(dy, u, x, w, col_scale=c, bias=bias, act="silu")
    n = [bool(v) for v in needs]
    got = bnd.dora_matmul_backward_int8(dy, u, x if n[1] else None, w if n[0] else None, col_scale=c, bias=bias,
                                        act="silu", need_dx=n[0], need_dw=n[1], need_dbias=n[2], need_dcol_scale=n[3])
    for need, g, f in zip(n, got, full):
        assert (g is not None) == need and (g is None or torch.equal(g, f))
    assert torch.equal(got[4], full[4])


@pytest.mark.parametrize("dtype,M,N,K", [("f32", 12, 20, 24), ("bf16", 70, 136, 200), ("f16", 300, 264, 72)])
def test_int8_backward_with_a_row_scale(dtype, M, N, K):
    rng, dy, u, x, w, c, bias = backward_case(M, N, K, dtype, 13, 32, 0, 64)
    rows = vec(rng, M, 0.4)
    got = bnd.dora_matmul_backward_int8(dy, u, x, w, row_scale=rows, col_scale=c, bias=bias, act="silu")
    check_backward(got, dy, u, x, w, c, bias, "silu", dtype, rows)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_int8_backward_without_rows_writes_its_sums(dtype):
    dt = TORCH_DT[dtype]
    stale = [torch.full((n,), float("nan"), device="cuda") for n in (8, 8, 8, 8, 128, 128)]
    del stale
    z8 = lambda *s: torch.empty(*s, dtype=torch.int8, device="cuda")   # noqa: E731
    e = torch.empty(0, device="cuda")
    w = bnd.Int8Rows(z8(8, 16).zero_(), torch.ones(8, device="cuda"))
    dx, dw, db, dc, du = bnd.dora_matmul_backward_int8(torch.empty(0, 8, dtype=dt, device="cuda"),
                                                       bnd.Int8Rows(z8(0, 8), e), bnd.Int8Rows(z8(0, 16), e), w)
    assert du.shape == (0, 8) and dx.shape == (0, 16)
    assert (db == 0).all() and (dc == 0).all() and (dw == 0).all()


def test_int8_gradients_against_differences():
    """fp32 gradients of a DoRA layer on an 8-bit base with packed u and x, of the values that the rows stand for."""
    rng = np.random.default_rng(13)
    M, N, K, r, s = 12, 20, 24, 8, 0.5
    (x8, xs), (w8, ws) = pack(rng, (M, K)), pack(rng, (N, K), 0.3)
    xr, wr = bnd.Int8Rows(x8, xs), bnd.Int8Rows(w8, ws)
    c, bias, dy = vec(rng, N), vec(rng, N, 0.3, 0.0), draw(rng, (M, N), "f32")
    _, u = bnd.dora_matmul_int8(x8, w8, xs, ws, col_scale=c, bias=bias, act="gelu", out_dtype=torch.float32, save=True)
    dx, dw, db, dc, du = bnd.dora_matmul_backward_int8(dy, u, xr, wr, col_scale=c, bias=bias, act="gelu")
    vals = dict(x=values(xr), w=values(wr), col_scale=host(c), bias=host(bias))
    grads = dict(x=host(dx), w=host(dw), col_scale=host(dc), bias=host(db))

    def loss(**kw):
        return (B.matmul(**{**vals, **kw}, name="gelu")[0] * host(dy)).sum()

    for k, g in grads.items():
        d, e = rng.standard_normal(g.shape), 1e-5
        num = (loss(**{k: vals[k] + e * d}) - loss(**{k: vals[k] - e * d})) / (2 * e)
        assert abs((g * d).sum() - num) <= 1e-4 * np.linalg.norm(g) * np.linalg.norm(d), k


# ---------------------------------------------------------------- as they are used together

def test_int8_graph_replays_and_streams():
    """Norm to int8 rows, integer product, packing, and both backward passes in one graph, replayed with eager work
    between, bitwise the eager results."""
    rng = np.random.default_rng(14)
    M, N, K, r = 96, 264, 528, 16
    o, _ = operands(M, N, K, r, "bf16", 14)
    x, res, nw, nb = draw(rng, (M, K), "bf16"), draw(rng, (M, K), "bf16"), vec(rng, K), vec(rng, K, 0.1, 0.0)
    dy = draw(rng, (M, N), "bf16")
    tail = {k: o[k] for k in ("col_scale", "bias")}

    def step():
        q, sc, h, mean, rstd = bnd.dora_layer_norm_quant(x, nw, nb, 1e-5, residual=res)
        y, u = bnd.dora_matmul_int8(**{**o, "x": q, "row_scale": sc}, act="silu", save=True)
        uq, us = bnd.dora_quantize_rows(u, group=64)
        dx, dw, db, dc, du = bnd.dora_matmul_backward_int8(dy, bnd.Int8Rows(uq, us, 64), bnd.Int8Rows(q, sc),
                                                           bnd.Int8Rows(o["w"], o["w_scale"]), act="silu", **tail)
        gx, gw, gb = bnd.dora_layer_norm_backward(dx, h, mean, rstd, nw)
        return q, y, u, uq, us, dx, dw, db, dc, gx, gw, gb, bnd.dora_dequantize_rows(uq, us, group=64)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [v.clone() for v in step()]
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        for g in got:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for g, v in zip(got, want):
            assert torch.equal(g, v)
        eager = step()
        torch.cuda.synchronize()
        for g, v in zip(eager, want):
            assert torch.equal(g, v)


def test_two_calls_at_once_on_two_streams():
    o, rng = operands(300, 520, 8208, 16, "bf16", 15)
    o2, _ = operands(300, 520, 8208, 16, "bf16", 16)
    want = [bnd.dora_matmul_int8(**v)[0] for v in (o, o2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[bnd.dora_matmul_int8(**v, stream=s)[0] for v, s in zip((o, o2), streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, want):
            assert torch.equal(g, w)


# Up to 16 tokens, whole steps of 128 and two blocks of 16 columns for a compute unit: one workgroup a unit walks them.
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,r", [(1, 12288, 2048, 0), (1, 12305, 2176, 8), (7, 12300, 8192, 512), (8, 16400, 2944, 40),
                                     (9, 8192, 8064, 0), (16, 28672, 256, 384), (16, 17000, 2176, 384), (13, 8207, 2048, 264), (12, 8192, 128, 64)])
def test_walking_kernel(M, N, K, r, out):
    o, rng = operands(M, N, K, 0 if out == "f32" else r, out, M + N + K)
    check(o, rng, out, ACTS[(M + N + K) % 5], M % 2 == 0, True)
    plain = {k: v for k, v in o.items() if k not in ("col_scale", "bias")}
    check(plain, rng, out, "none", False, False)


def test_products_beside_the_walking_kernel():
    """What it does not take: a depth of no whole steps, one past 8192, a pair of no whole chunks or past a step a wave."""
    for M, N, K, r in ((3, 8192, 1000, 16), (3, 8192, 8320, 16), (16, 8192, 1024, 20), (16, 8192, 1024, 520),
                       (16, 8176, 1024, 16), (17, 8192, 1024, 16)):
        o, rng = operands(M, N, K, r, "bf16", M + N + K)
        check(o, rng, "bf16", "silu", True, False)


# Up to 32 rows that go to the tiles: 17 and more over many columns, fewer over the most at shallow depths or past the
# walking kernel's, with a split depth, a pair off the 16-byte grid, and one row.
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,r", [(17, 8200, 1040, 20), (32, 12288, 4096, 384), (24, 4112, 8208, 0), (3, 16400, 2048, 16),
                                     (1, 16384, 16, 0), (16, 20001, 272, 5), (14, 8208, 16400, 40)])
def test_few_rows_in_tiles(M, N, K, r, out):
    r = 0 if out == "f32" else r
    assert bnd.dora_matmul_int8_plan_info(M, N, K, r)["tile_rows"] > 0
    o, rng = operands(M, N, K, r, out, M + N + K)
    check(o, rng, out, ACTS[(M + N + K) % 5], M % 2 == 0, True)


# Small tiles on rows at any address: ends of every length in a row's last chunk, of x and w or the pair alone, one stage
# and many, a split depth, the shortest rows, and results off 16 bytes.
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,r", [(333, 1001, 777, 24), (65, 700, 16, 8), (70, 900, 17, 9), (300, 520, 8189, 0),
                                     (64, 8192, 1025, 77), (40, 5000, 127, 63), (257, 321, 128, 13), (400, 300, 255, 130),
                                     (33, 4111, 784, 500), (1000, 1000, 1001, 11), (129, 777, 31, 15)]
                         + [(100, 1000, 256 + e, 0) for e in range(1, 16)])
def test_tiles_on_rows_at_any_address(M, N, K, r, out):
    r = 0 if out == "f32" else r
    o, rng = operands(M, N, K, r, out, M + N + K)
    check(o, rng, out, ACTS[(M + N + K) % 5], M % 2 == 0, True)


def test_tiles_at_any_address_stay_in_their_rows():
    """Operands off 16 bytes inside larger buffers whose other bytes would show; the same values from aligned ones."""
    rng = np.random.default_rng(36)
    M, N, K, r = 100, 333, 640, 16
    o, _ = operands(M, N, K, r, "bf16", 36)

    def inside(t, by):
        buf = torch.full((t.numel() + 64,), 77, device="cuda", dtype=t.dtype)
        buf[by:by + t.numel()] = t.flatten()
        return buf[by:by + t.numel()].view(t.shape)

    want, _ = bnd.dora_matmul_int8(**o)
    moved = {k: inside(v, 3) if k in ("x", "w", "t", "b") else v for k, v in o.items()}
    got, _ = bnd.dora_matmul_int8(**moved)
    assert torch.equal(got, want)
    x, w, xs, ws = (torch.ones(s, device="cuda", dtype=d) for s, d in (((100, 300), torch.int8), ((333, 300), torch.int8),
                                                                     ((100,), torch.float32), ((333,), torch.float32)))
    y, _ = bnd.dora_matmul_int8(inside(x, 5), inside(w, 9), xs, ws, out_dtype=torch.float32)
    assert (y == 300).all()


def aligned_rows(rng, shape, dtype, group):
    v = draw(rng, shape, dtype)
    return bnd.Int8Rows(*bnd.dora_quantize_rows(v, group=group), group)


# (M, N, K) whose products take the tiles of 256 and 128 rows: rows in whole chunks of 16 bytes, which these kernels
# read as they are held; odd row counts, ends inside a tile, a split depth, and depths of one stage and less.
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,group", [(8200, 384, 4112, 128), (4100, 2056, 4112, 0), (2077, 1021, 2064, 64), (8192, 64, 2048, 32),
                                         (1021, 4104, 4112, 256), (5000, 100, 8192, 0), (16384, 40, 1040, 128),
                                         (130, 1000, 8208, 32), (1000, 8200, 2048, 0), (600, 600, 28672, 64)])
def test_products_that_read_int8_rows(M, N, K, group, dtype):
    rng = np.random.default_rng(M + N)
    dy, u = draw(rng, (M, N), dtype), draw(rng, (M, N), dtype)
    x, w, c = aligned_rows(rng, (M, K), dtype, group), aligned_rows(rng, (N, K), dtype, group), vec(rng, N, 0.2)
    got = bnd.dora_matmul_backward_int8(dy, u, x, w, col_scale=c)
    check_backward(got, dy, u, x, w, c, torch.zeros(N, device="cuda"), "none", dtype)
    again = bnd.dora_matmul_backward_int8(dy, u, x, w, col_scale=c)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("at", ["x", "w"])
def test_int8_rows_off_the_grid(at):
    """q one byte into its buffer: the same values from copies as from the rows themselves, but for how sums are ordered."""
    rng = np.random.default_rng(31)
    M, N, K = 2100, 520, 2064
    dy, u = draw(rng, (M, N), "bf16"), draw(rng, (M, N), "bf16")
    v = {"x": aligned_rows(rng, (M, K), "bf16", 128), "w": aligned_rows(rng, (N, K), "bf16", 0)}
    v[at] = v[at]._replace(q=off(v[at].q))
    got = bnd.dora_matmul_backward_int8(dy, u, v["x"], v["w"])
    check_backward(got, dy, u, v["x"], v["w"], torch.ones(N, device="cuda"), torch.zeros(N, device="cuda"), "none", "bf16")


def test_int8_rows_with_a_nan_scale_reach_their_own():
    rng = np.random.default_rng(32)
    M, N, K = 2100, 384, 4096
    dy, u = draw(rng, (M, N), "bf16"), draw(rng, (M, N), "bf16")
    x = aligned_rows(rng, (M, K), "bf16", 128)
    clean = bnd.dora_matmul_backward_int8(dy, u, x, None, need_dx=False)[1]
    x.scale[2099, 3] = float("nan")
    x.q[2099, 3 * 128:4 * 128] = 0
    dw = bnd.dora_matmul_backward_int8(dy, u, x, None, need_dx=False)[1]
    assert torch.isnan(dw[:, 384:512]).all()
    keep = [k for k in range(K) if not 384 <= k < 512]
    assert torch.equal(dw[:, keep], clean[:, keep])


def test_the_largest_values_that_int8_rows_stand_for():
    x = torch.zeros(4, 4096, device="cuda", dtype=torch.bfloat16)
    x[:, ::3], x[:, 1::3] = 3.38e38, -3.38e38
    q, s = bnd.dora_quantize_rows(x, group=128)
    back = bnd.dora_dequantize_rows(q, s, group=128)
    assert torch.isfinite(back).all() and (back.float() / x.float().where(x != 0, back.float()) - 1)[:, ::3].abs().max() < 2.0 ** -7
    dy = torch.zeros(4096, 384, device="cuda", dtype=torch.bfloat16)
    dy[1] = 2.0 ** -20
    rows = bnd.Int8Rows(q.repeat(1024, 1), s.repeat(1024, 1), 128)
    dw = bnd.dora_matmul_backward_int8(dy, dy, rows, None, need_dx=False)[1]
    assert torch.equal(dw, (back[1].float() * 2.0 ** -20).bfloat16().expand(384, 4096))


def test_backward_offsets_past_32_bits():
    """x8 of more than 2^32 bytes, read as it is held and (one byte off) from a copy, and u8 of as many."""
    M, N, K, n = 2100000, 384, 2064, 70
    rng = np.random.default_rng(33)
    x = bnd.Int8Rows(torch.zeros(M, K, device="cuda", dtype=torch.int8), torch.ones(M, 17, device="cuda"), 128)
    tail = aligned_rows(rng, (n, K), "bf16", 128)
    x.q[-n:], x.scale[-n:] = tail.q, tail.scale
    dy = torch.zeros(M, N, device="cuda", dtype=torch.bfloat16)
    dy[-n:] = draw(rng, (n, N), "bf16")
    got = bnd.dora_matmul_backward_int8(dy, dy, x, None, need_dx=False)
    one, zero = torch.ones(N, device="cuda"), torch.zeros(N, device="cuda")
    short = [got[0], got[1], got[2], got[3], got[4][-n:]]
    check_backward(short, dy[-n:], dy[-n:], tail, tail.q.new_zeros(N, K).bfloat16(), one, zero, "none", "bf16")
    assert not got[4][:-n].any()
    moved = x._replace(q=off(x.q))
    del x
    again = bnd.dora_matmul_backward_int8(dy, dy, moved, None, need_dx=False)
    check_backward([None, again[1], again[2], again[3], again[4][-n:]], dy[-n:], dy[-n:], tail,
                   tail.q.new_zeros(N, K).bfloat16(), one, zero, "none", "bf16")
    # u8: the same rows, of K columns
    big = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    big[-n:] = draw(rng, (n, K), "bf16")
    _, _, db, dc, du = bnd.dora_matmul_backward_int8(big, moved, None, None, act="silu", need_dx=False, need_dw=False)
    c1, c0 = torch.ones(K, device="cuda"), torch.zeros(K, device="cuda")
    check_backward([None, None, db, dc, du[-n:]], big[-n:], tail, tail.q.new_zeros(n, 8).bfloat16(),
                   tail.q.new_zeros(K, 8).bfloat16(), c1, c0, "silu", "bf16")
    assert not du[:-n].any()


def test_transposed_copies_of_more_tiles_than_workgroups():
    """Rows whose fp32 copies are more 64 x 64 tiles than one launch has workgroups for them."""
    M, K, n = 2000070, 130, 150
    rng = np.random.default_rng(35)
    x = bnd.Int8Rows(torch.randint(-127, 128, (M, K), device="cuda", dtype=torch.int8), torch.full((M,), 0.25, device="cuda"))
    u = bnd.Int8Rows(x.q[:, :1].contiguous(), x.scale)
    at = torch.randint(0, M, (n,), device="cuda").unique()
    dy = torch.zeros(M, 1, device="cuda")
    dy[at] = torch.from_numpy(rng.integers(-4, 5, (len(at), 1)).astype(np.float32)).cuda()
    w = bnd.Int8Rows(torch.randint(-127, 128, (1, K), device="cuda", dtype=torch.int8), torch.full((1,), 0.5, device="cuda"))
    dx, dw, db, dc, du = bnd.dora_matmul_backward_int8(dy, u, x, w)
    # (whole numbers times powers of two: every sum is exact)
    want = (dy[at] * x.q[at].float() * 0.25).sum(0, keepdim=True)
    assert torch.equal(du, dy) and torch.equal(dx, dy * (w.q.float() * 0.5))
    assert torch.equal(dw, want) and dc.item() == want[0, 0].item() and db.item() == dy.sum().item()


@pytest.mark.parametrize("M,N,K", [(0, 384, 4096), (8200, 0, 4096), (8200, 384, 0)])
def test_empty_int8_backward(M, N, K):
    dt, i8 = torch.bfloat16, torch.int8
    rows = lambda a, b: bnd.Int8Rows(torch.ones(a, b, device="cuda", dtype=i8), torch.ones(a, device="cuda"))   # noqa: E731
    dx, dw, db, dc, du = bnd.dora_matmul_backward_int8(torch.ones(M, N, device="cuda", dtype=dt), rows(M, N), rows(M, K),
                                                       rows(N, K))
    assert dx.shape == (M, K) and dw.shape == (N, K) and du.shape == (M, N)
    assert (dx == 0).all() and (dw == 0).all()
    if M == 0:
        assert (db == 0).all() and (dc == 0).all()


def test_du_in_the_place_of_dy():
    """The C entry allows du to be dy itself (rows are asked for ahead of the ones being written)."""
    rng = np.random.default_rng(34)
    M, N = 1000, 520
    dy = draw(rng, (M, N), "bf16")
    u = aligned_rows(rng, (M, N), "bf16", 64)
    want = bnd.dora_matmul_backward_int8(dy, u, None, None, act="gelu", need_dx=False, need_dw=False)
    need = bnd.dora_matmul_backward_int8_workspace_size(M, N, 0, "bf16", bnd.GRAD_SUMS + bnd.GRAD_DU + bnd.GRAD_ALIGNED, 0)
    ws = torch.empty(need, device="cuda", dtype=torch.uint8)
    db, dc, into = torch.empty(N, device="cuda"), torch.empty(N, device="cuda"), dy.clone()
    arg = bnd._Int8RowsArg(u.q.data_ptr(), u.scale.data_ptr(), 64)
    import ctypes
    bnd._call("dora_matmul_backward_int8", into.data_ptr(), None, ctypes.byref(arg), None, None, None, None, 0, M, N, 0,
              None, None, None, 2, into.data_ptr(), None, None, db.data_ptr(), dc.data_ptr(), ws.data_ptr(), need,
              torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(into, want[4]) and torch.equal(db, want[2]) and torch.equal(dc, want[3])
