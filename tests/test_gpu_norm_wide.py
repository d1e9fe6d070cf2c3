"""Weight gradients of rows so wide that one workgroup for every 64 columns would pass a launch's 2^32 threads."""

import pytest
import torch

from dora_weight_norm_amd import binding as bnd

pytestmark = pytest.mark.gpu


def rows(T, d):
    gen = torch.Generator(device="cuda").manual_seed(d)
    return (torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))


def off(got, want, sizes):
    """The most by which got is off, in 2^-24 of sizes (two roundings of a factor and two of the product: 4)."""
    return ((got - want).abs() / (sizes + 1e-30)).max().item() * 2 ** 24


# 2 d columns: past 2^32 threads, and not at the end of a block of columns or of a wave's share of one
@pytest.mark.parametrize("d", [(1 << 27) - 3, (1 << 27) + 70])
def test_layer_norm_backward_of_one_wide_row(d):
    dy, h = rows(1, d)
    mean, rstd = torch.full((1,), 0.25, device="cuda"), torch.full((1,), 0.75, device="cuda")
    _, dw, db = bnd.dora_layer_norm_backward(dy, h, mean, rstd, None)
    assert torch.equal(db, dy[0].float())
    want = dy[0].double() * ((h[0].double() - 0.25) * 0.75)
    assert off(dw, want, want.abs()) <= 4
    del want
    z, e = torch.empty(0, d, device="cuda", dtype=torch.bfloat16), torch.empty(0, device="cuda")
    dw.fill_(1), db.fill_(1)
    bnd.dora_layer_norm_backward(z, z, e, e, None, dweight=dw, dbias=db)
    assert not dw.any() and not db.any()


def test_rms_norm_backward_of_one_wide_row():
    d = (1 << 28) + 70
    dy, h = rows(1, d)
    rstd = torch.full((1,), 0.75, device="cuda")
    _, dw = bnd.dora_rms_norm_backward(dy, h, rstd, None, need_dweight=True)
    want = dy[0].double() * (h[0].double() * 0.75)
    assert off(dw, want, want.abs()) <= 4
