"""The integer product's kernels on operands that decide which of them runs; bounds as in test_gpu_int8.py."""

import numpy as np
import pytest
import torch

from block_helpers import draw
from dora_weight_norm_amd import binding as bnd
from test_gpu_int8 import ACTS, aligned_rows, check, off, operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,r", [(32, 20000, 8192, 20), (17, 20001, 8208, 384), (14, 20000, 8320, 0), (24, 28672, 8192, 5),
                                     (1, 28672, 1024, 3), (64, 20000, 8192, 1), (33, 20001, 8189, 7), (50, 4112, 28672, 8)])
@pytest.mark.parametrize("at", ["x", "w", "xwtb"])
def test_one_row_of_tiles_takes_no_copy_of_w(M, N, K, r, at):
    """Operands one element off the 16-byte grid, and pairs whose rows are shorter than its step."""
    al = 15 - sum(1 << i for i, k in enumerate("xwtb") if k in at)
    p = bnd.dora_matmul_int8_plan_info(M, N, K, r, aligned_operands=al)
    assert p["tile_rows"] > 0 and p["copies"] & 2 == 0, p
    o, rng = operands(M, N, K, r, "bf16", M + N)
    o = {k: off(v) if k in at and isinstance(v, torch.Tensor) else v for k, v in o.items()}
    check(o, rng, "bf16", ACTS[M % 5], M % 2 == 0, True)
    y = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    bnd.dora_matmul_int8(**o, y=y)
    assert torch.cuda.max_memory_allocated() - before < N * K // 2


@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,r", [(16, 16000, 256, 384), (16, 16383, 2048, 512), (9, 12289, 128, 8), (1, 12288, 8192, 512)])
def test_walking_kernel_with_a_pair(M, N, K, r, out):
    assert bnd.dora_matmul_int8_plan_info(M, N, K, r)["kernel"] == "walk"
    o, rng = operands(M, N, K, r, out, M + N + K)
    check(o, rng, out, ACTS[(M + N) % 5], M % 2 == 0, True)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,r", [(300, 333, 640, 16), (300, 333, 640, 0), (128, 8192, 512, 384), (64, 2000, 8192, 16),
                                     (64, 20000, 1024, 8), (257, 1001, 16, 8)])
def test_tiles_at_any_address_give_the_other_tiles_results(M, N, K, r, out):
    """To the bit, from operands inside larger buffers whose other bytes would show."""
    r = 0 if out == "f32" else r
    plans = [bnd.dora_matmul_int8_plan_info(M, N, K, r, aligned_operands=al) for al in (15, 0)]
    assert [p["kernel"] for p in plans] == ["tiles", "tiles_anywhere"] and plans[0]["tile_rows"] == 64
    assert plans[0]["splits"] == plans[1]["splits"]
    o, rng = operands(M, N, K, r, out, 36)
    res = rng.standard_normal((M, N))
    res = torch.from_numpy(res).cuda().to({"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[out])

    def inside(t, by):
        buf = torch.full((t.numel() + 64,), 77, device="cuda", dtype=t.dtype)
        buf[by:by + t.numel()] = t.flatten()
        return buf[by:by + t.numel()].view(t.shape)

    want = bnd.dora_matmul_int8(**o, residual=res, act="silu", save=True, out_dtype=res.dtype)
    moved = {k: inside(v, 3) if k in ("x", "w", "t", "b") else v for k, v in o.items()}
    got = bnd.dora_matmul_int8(**moved, residual=res, act="silu", save=True, out_dtype=res.dtype)
    for g, w in zip(got, want):
        assert torch.equal(g, w)


# Depths in parts on tiles of 128 and of 256 rows, and one part.
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,group,rows", [(8200, 384, 4112, 128, 128), (8192, 384, 8192, 32, 256), (4100, 2056, 4112, 256, 256),
                                              (2077, 1021, 2064, 64, 128)])
def test_bad_scales_of_held_rows_reach_their_own(M, N, K, group, rows, dtype, bad):
    """A scale that is no number, of rows that the tiles turn into 16 bits themselves: in the columns of its group, of
    every row of the result, and nowhere else."""
    p = bnd.dora_matmul_backward_int8_plan_info(M, N, K, dtype)
    assert p["dw"]["reads"] == "int8_rows" and p["dw"]["tile_rows"] == rows and p["dx"]["reads"] == "int8_rows", p
    rng = np.random.default_rng(32)
    dy, u = draw(rng, (M, N), dtype), draw(rng, (M, N), dtype)
    x, w = aligned_rows(rng, (M, K), dtype, group), aligned_rows(rng, (N, K), dtype, group)
    clean = bnd.dora_matmul_backward_int8(dy, u, x, w)
    last = (K - 1) // group
    for rows8, row, g in ((x, M - 1, 3), (x, 5, last), (w, N - 1, 2)):
        rows8.scale[row, g] = bad
        rows8.q[row, g * group:(g + 1) * group] = 0
    got = bnd.dora_matmul_backward_int8(dy, u, x, w)
    for i, groups in ((0, (2,)), (1, (3, last))):
        keep = torch.ones(K, dtype=torch.bool, device="cuda")
        for g in groups:
            keep[g * group:(g + 1) * group] = False
        assert torch.isnan(got[i][:, ~keep]).all(), i
        # (the other values of the rows that turned bad are as before)
        assert torch.equal(got[i][:, keep], clean[i][:, keep]), i
