"""Plans of the integer product for operands at any address (no GPU: queries alone)."""

import ctypes
import os

import pytest
import torch

from dora_weight_norm_amd import binding as bnd

pytestmark = pytest.mark.skipif(not os.path.exists(bnd.LIB_PATH), reason="libdora.so not built")

# few rows that tiles take where w lies on the 16-byte grid
FEW_IN_TILES = [(32, 28672, 8192, 0), (17, 28672, 8192, 384), (16, 28672, 2048, 0), (1, 28672, 1024, 8),
                (14, 28672, 8320, 0), (32, 20000, 4096, 20), (24, 28672, 8192, 5)]


@pytest.mark.parametrize("M,N,K,r", FEW_IN_TILES)
@pytest.mark.parametrize("al", range(16))
def test_w_off_the_grid_is_not_copied_for_few_rows(M, N, K, r, al):
    p = bnd.dora_matmul_int8_plan_info(M, N, K, r, aligned_operands=al)
    assert p["tile_rows"] > 0 and p["copies"] & 2 == 0, p


@pytest.mark.parametrize("M,N,K,r", [(64, 28672, 8192, 0), (33, 28672, 8189, 24), (64, 100000, 2000, 5), (40, 300, 17, 3)])
def test_w_off_the_grid_is_not_copied_for_one_row_of_tiles(M, N, K, r):
    for al in (0, 13):
        p = bnd.dora_matmul_int8_plan_info(M, N, K, r, aligned_operands=al)
        assert p["tile_rows"] == 64 and p["copies"] & 2 == 0, p
    assert bnd.dora_matmul_int8_plan_info(128, 28672, 8192, 0, aligned_operands=13)["copies"] == 2


@pytest.mark.parametrize("M,N,K,r", FEW_IN_TILES + [(17, 8200, 1040, 20), (24, 4112, 8208, 0), (16, 20001, 272, 5),
                                                    (32, 8192, 8192, 384), (16, 8192, 16400, 40), (32, 2048, 16384, 0),
                                                    (64, 28672, 8192, 5), (33, 28672, 8189, 24), (50, 28672, 8192, 384)])
def test_a_workspace_for_few_rows_at_any_address_serves_them_at_all(M, N, K, r):
    sizes = [bnd.dora_matmul_int8_workspace_size(M, N, K, r, al) for al in range(16)]
    assert max(sizes) == sizes[0] and max(sizes) < N * K // 2     # (no room for a copy of w)
    for al in range(16):                                           # s = 0 reads no pair
        assert bnd.dora_matmul_int8_workspace_size(M, N, K, 0, al) <= sizes[al]


@pytest.mark.parametrize("kernel,shapes", [
    ("walk", [(1, 12288, 2048, 0), (7, 12300, 8192, 512), (9, 8192, 8064, 0), (16, 16000, 256, 384), (12, 8192, 128, 64)]),
    ("few_rows", [(1, 8192, 8192, 0), (16, 8192, 8320, 16), (16, 8192, 1024, 520), (32, 1024, 4096, 0), (100, 333, 640, 16)]),
    ("tiles", [(16, 28672, 256, 384), (32, 28672, 8192, 0), (300, 333, 640, 16), (8192, 8192, 8192, 384)]),
    ("tiles_anywhere", [(333, 1001, 777, 24), (40, 5000, 127, 63), (300, 333, 640, 13), (64, 28672, 8189, 0)]),
    (None, [(0, 64, 64, 0), (64, 0, 64, 0)])])
def test_kernels_of_shapes(kernel, shapes):
    for a in shapes:
        assert bnd.dora_matmul_int8_plan_info(*a)["kernel"] == kernel, a


def test_the_plain_products_plan_names_no_kernel():
    buf = (ctypes.c_int64 * 8)()
    assert bnd.load().dora_matmul_plan_info(300, 333, 640, 16, 0, 15, buf, 8) == 0 and list(buf)[5:] == [-1] * 3
    assert bnd.load().dora_matmul_int8_plan_info(300, 333, 640, 16, 15, buf, 8) == 0 and list(buf)[5:] == [0, -1, -1]


def test_backward_plans():
    plan = bnd.dora_matmul_backward_int8_plan_info
    p = plan(8200, 384, 4112, "bf16")
    assert p["dw"] == {"tile_rows": 128, "splits": 5, "reads": "int8_rows"} and p["dx"]["reads"] == "int8_rows"
    assert plan(8192, 384, 8192, "f16")["dw"]["tile_rows"] == 256
    assert plan(2100, 384, 4096, "bf16")["dw"] == {"tile_rows": 64, "splits": 1, "reads": "copy"}
    for a in ((8192, 8192, 8192, "bf16"), (2100, 520, 2064, "bf16", 15), (64, 128, 256, "f32")):   # deep, off the grid, fp32
        p = plan(*a)
        assert p["dx"]["reads"] == p["dw"]["reads"] == "copy", a
    p = plan(4096, 4096, 4096, "bf16", bnd.GRAD_DX + bnd.GRAD_DW + bnd.GRAD_ALIGNED, 32, 0)
    assert p["dx"]["reads"] == "as_given" and p["dw"]["reads"] == "int8_rows"
    p = plan(4096, 4096, 4096, "bf16", bnd.GRAD_DW, 0, 0)
    assert p["dx"] is None and p["dw"]["reads"] == "copy"
    p = plan(0, 64, 64, "bf16")
    assert p["dx"] is None and p["dw"] is not None
    assert p["workspace_bytes"] == bnd.dora_matmul_backward_int8_workspace_size(0, 64, 64, "bf16")
    f, buf = bnd.load().dora_matmul_backward_int8_plan_info, (ctypes.c_int64 * 9)()
    assert f(64, 64, 64, 0, 31, 1, 1, buf, 9) == 0 and list(buf)[7:] == [-1, -1]
    assert f(64, 64, 64, 0, 31, 1, 1, None, 7) == 1 and f(64, 64, 64, 0, 31, 1, 1, buf, -1) == 1
    assert f(64, 64, 64, 3, 31, 1, 1, buf, 7) == 2 and f(64, 64, 64, 0, 32, 1, 1, buf, 7) == 1
    assert f(-1, 1, 1, 0, 31, 1, 1, buf, 7) == 1 and f(64, 64, 64, 0, 31, -1, 1, buf, 7) == 1


@pytest.mark.parametrize("M,N,K", [(64, 128, 256), (8192, 8192, 4096), (333, 1001, 777), (8200, 384, 4112), (1, 1, 1), (64, 64, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_backward_workspaces(M, N, K, dtype):
    """Of one scale a row at least those of several and of none beside the copies that these take; an operand of its own
    for each product of 16-bit types with one scale a row."""
    def need(outputs, x, w):
        return bnd._size_of("dora_matmul_backward_int8_scales_workspace_size", M, N, K, bnd._dtype_code(dtype), outputs, x, w)

    for outputs in range(32):
        whole = bnd.dora_matmul_backward_int8_workspace_size(M, N, K, dtype, outputs, bnd.HELD_X + bnd.HELD_W)
        assert whole == need(outputs, 1, 1) == max(need(outputs, x, w) for x in (1, 5) for w in (1, 5))
        for held in range(4):
            x, w = held & 1, held >> 1
            assert bnd.dora_matmul_backward_int8_workspace_size(M, N, K, dtype, outputs, held) == need(outputs, x, w)
    du = M * N * 2
    alone = bnd.GRAD_DX + bnd.GRAD_DU + bnd.GRAD_ALIGNED
    if dtype != "f32" and N % 8 == 0 and K > 0:
        assert need(alone, 0, 1) - need(alone, 0, 5) >= du
    sz = ctypes.c_size_t()
    f = bnd.load().dora_matmul_backward_int8_scales_workspace_size
    assert f(M, N, K, 0, 31, 1, 1, None) == 1 and f(M, N, K, 0, 31, 1, -1, ctypes.byref(sz)) == 1


@pytest.mark.parametrize("q_dtype", [None, torch.uint8, torch.bfloat16, "int8"])
def test_the_norms_8_bit_type_is_one_of_two(q_dtype):
    with pytest.raises(TypeError, match="q_dtype"):
        bnd.dora_layer_norm_quant(torch.zeros(4, 8), None, None, 1e-5, q_dtype=q_dtype, y=torch.zeros(4, 8))
