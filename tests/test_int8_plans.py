"""Plans of the integer product for operands at any address (no GPU: queries alone)."""

import os

import pytest

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
