"""The calls on int8 rows and the layer norm launch on the tensors' GPU when another one is current (no GPU: stand-ins)."""

import torch

from dora_weight_norm_amd import binding as bnd
from test_binding_device import OnGpu1, gpus  # noqa: F401  (the fixture)


def test_calls_on_int8_rows_set_the_tensors_gpu(gpus):  # noqa: F811
    calls, current = gpus
    i8 = torch.int8
    x, v, t = OnGpu1((4, 8)), OnGpu1((8,)), OnGpu1((4,))
    q, w = OnGpu1((4, 8), i8), OnGpu1((6, 8), i8)
    bnd.dora_layer_norm(x, v, v, 1e-6)
    bnd.dora_layer_norm_quant(x, v, v, 1e-6, residual=x)
    bnd.dora_layer_norm_backward(x, x, t, t, v)
    bnd.dora_quantize_rows(x)
    bnd.dora_quantize_rows(x, group=32)
    bnd.dora_dequantize_rows(q, t)
    bnd.dora_matmul_int8(q, w, t, OnGpu1((6,)))
    bnd.dora_matmul_backward_int8(OnGpu1((4, 6)), bnd.Int8Rows(OnGpu1((4, 6), i8), t), bnd.Int8Rows(q, t),
                                  bnd.Int8Rows(w, OnGpu1((6,))))
    assert len(calls) == 8 and all(dev == 1 for _, dev in calls), calls
    assert current == [0]
