"""The binding launches on the tensors' GPU when another one is current (no GPU: the library and the tensors are stand-ins)."""

import contextlib

import pytest
import torch

from dora_weight_norm_amd import binding as bnd


class OnGpu1:
    """What the binding asks of a tensor, of one that lives on cuda:1."""

    def __init__(self, shape, dtype=torch.float32):
        self.shape, self.dtype, self.is_cuda = torch.Size(shape), dtype, True

    def get_device(self):
        return 1

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def gpus(monkeypatch):
    """Two GPUs with the first current; a list of (call, GPU that is current then)."""
    calls, current = [], [0]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], getattr(d, "index", d)
        yield
        current[0] = before

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, current[0])) or 0

    monkeypatch.setattr(bnd, "_lib", Lib())
    monkeypatch.setattr(bnd, "_current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(bnd, "_current_raw_stream", lambda dev: 0)
    monkeypatch.setattr(bnd, "_size_of", lambda *a: 0)
    monkeypatch.setattr(bnd, "_new", lambda stream, shape, dtype, dev: OnGpu1(shape, dtype))
    monkeypatch.setattr(torch.cuda, "device", device)
    return calls, current


def test_calls_of_the_block_set_the_tensors_gpu(gpus):
    calls, current = gpus
    x, w, v = OnGpu1((4, 8)), OnGpu1((6, 8)), OnGpu1((8,))
    bnd.dora_rms_norm(x, v, 1e-6)
    bnd.dora_rms_norm_backward(x, x, OnGpu1((4,)), v)
    bnd.dora_matmul(x, w)
    bnd.dora_matmul_backward(OnGpu1((4, 6)), OnGpu1((4, 6)), x, w)
    assert len(calls) == 4 and all(dev == 1 for _, dev in calls), calls
    assert current == [0]
    current[0] = 1
    bnd.dora_matmul(x, w)
    assert calls[-1][1] == 1


def test_calls_of_the_norm_and_compose_set_the_tensors_gpu(gpus):
    _, current = gpus
    with bnd._on(None, torch.device("cuda", 1)):
        assert current == [1]
    assert current == [0]
    with bnd._on(None, torch.device("cuda", 0)):
        assert current == [0]
