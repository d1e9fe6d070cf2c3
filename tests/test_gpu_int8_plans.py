"""The integer product's kernels on operands that decide which of them runs; bounds as in test_gpu_int8.py."""

import pytest
import torch

from dora_weight_norm_amd import binding as bnd
from test_gpu_int8 import ACTS, check, off, operands

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
