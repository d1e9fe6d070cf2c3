"""The row norm of a layer on an 8-bit base beside that of the values which its product multiplies.

Tolerance: ||V16 + L|| - ||V + L|| is at most ||V16 - V||, half a step (2^-8, 2^-11 of a value, 2^-25 of fp16's
subnormal ones) of the row norm of V; 1e-5 of the norm is the norm call's own.
"""

import numpy as np
import pytest
import torch

from block_helpers import HALF, TINY, host
from dora_weight_norm_amd import block
from oracle import int8_oracle as Q
from test_gpu_block import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,f,r", [("bf16", 512, 1024, 16), ("f16", 512, 1024, 16), ("bf16", 4096, 512, 64),
                                         ("f16", 777, 130, 5), ("bf16", 8192, 384, 384)])
def test_row_norm_of_an_8_bit_base(dtype, d, f, r):
    p, _ = make(dtype, d, f, r)
    for layer in (block.int8_base(p.up), block.int8_base(p.down)):
        V = Q.dequantize_rows(host(layer.W.q), host(layer.W.scale))
        want = np.linalg.norm(V + layer.s * host(layer.B) @ host(layer.A), axis=1)
        wn, g = layer.magnitude()
        tol = HALF[dtype] * np.linalg.norm(V, axis=1) + TINY[dtype] * V.shape[1] ** 0.5 + 1e-5 * want
        assert (np.abs(host(wn) - want) <= tol).all()
        assert (np.abs(host(g) * host(wn) - host(layer.m)) <= 1e-6 * np.abs(host(layer.m))).all()
        # the norm of the values in 16 bits, to the bit that of a layer that holds them
        same = block.AdaptedLayer(layer.weight(), layer.A, layer.B, layer.m, layer.s)
        assert torch.equal(same.magnitude()[0], wn)
