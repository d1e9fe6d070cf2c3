"""Scales of int8 rows on the GPU: the fp32 quotient of the largest value and 127 to the bit, by numpy's division."""

import numpy as np
import pytest
import torch

from block_helpers import TORCH_DT, draw, host, vec
from dora_weight_norm_amd import binding as bnd

pytestmark = pytest.mark.gpu
GROUPS = [0, 32, 64, 128, 256]


def quotient(top):
    return np.asarray(top, np.float32) / np.float32(127)


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_half_of_every_short_maximum(dtype, group):
    """Maxima of eight significant bits, with half of each beside them, which lies on or beside the border of 63 and 64."""
    top = np.repeat(1 + np.arange(128) / 128, 3) * np.tile([1, 2.0 ** -5, 2.0 ** 9], 128)
    x = np.zeros((len(top), 256))
    x[:, 7::32], x[:, 20::32], x[:, 31::32] = top[:, None], -top[:, None] / 2, top[:, None] / 4
    t = torch.from_numpy(x.astype(np.float32)).cuda().to(TORCH_DT[dtype])
    assert np.array_equal(host(t), x)
    q, s = bnd.dora_quantize_rows(t, group=group)
    want = quotient(top)
    assert np.array_equal(s.cpu().numpy().reshape(len(top), -1), np.repeat(want[:, None], s.numel() // len(top), 1))
    assert np.array_equal(host(q), np.rint(x / want.astype(np.float64)[:, None]))


@pytest.mark.parametrize("T,d,group", [(4096, 64, 0), (4096, 256, 32), (300, 1024, 128), (40, 20000, 0), (3, 4096, 256)])
def test_maxima_of_all_sizes(T, d, group):
    rng = np.random.default_rng(42)
    x = rng.standard_normal((T, d)) * np.exp(rng.uniform(-62, 84, (T, 1)))
    x = torch.from_numpy(x.astype(np.float32)).cuda()
    g = group or d
    top = np.stack([np.abs(x.cpu().numpy()[:, k:k + g]).max(1) for k in range(0, d, g)], 1)
    _, s = bnd.dora_quantize_rows(x, group=group)
    assert np.array_equal(s.cpu().numpy().reshape(top.shape), np.maximum(quotient(top), np.float32(2.0 ** -100)))


@pytest.mark.parametrize("T,d", [(1, 64), (700, 1000), (5, 8192), (3, 20000)])
def test_scales_of_the_layer_norms_rows(T, d):
    """fp32 rows, whose y is the value that the scale is taken of."""
    rng = np.random.default_rng(43)
    x, y = draw(rng, (T, d), "f32"), torch.empty(T, d, device="cuda")
    _, s, _, _, _ = bnd.dora_layer_norm_quant(x, vec(rng, d), vec(rng, d, 0.1, 0.0), 1e-5, y=y)
    assert np.array_equal(s.cpu().numpy(), quotient(np.abs(y.cpu().numpy()).max(1)))
