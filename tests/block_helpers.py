"""Inputs and derived bounds of the norm and product tests."""

import numpy as np
import torch

TORCH_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
EPS32 = 2.0 ** -24
# half a step of the storage type relative to a value, and half its smallest step
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": EPS32}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}


def draw(rng, shape, dtype, std=1.0, mean=0.0):
    """A device tensor of the storage type."""
    v = torch.from_numpy((rng.standard_normal(shape) * std + mean).astype(np.float32))
    return v.cuda().to(TORCH_DT[dtype])


def vec(rng, n, std=0.1, mean=1.0):
    return torch.from_numpy((rng.standard_normal(n) * std + mean).astype(np.float32)).cuda()


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, ref, tol, what):
    """|got - ref| <= tol everywhere; NaN and infinities in the same places."""
    got = host(got)
    ref = np.asarray(ref, np.float64)
    assert got.shape == ref.shape, what
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), what
    tol = np.broadcast_to(tol, ref.shape)
    err = np.abs(got - ref)[fine]
    bad = err > tol[fine]
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(err / np.maximum(tol[fine], 1e-300)):.2f}x"


def rounded(dtype, ref, fp32_err):
    """Tolerance of a value rounded once to `dtype` that was computed with an error of fp32_err."""
    return HALF[dtype] * (np.abs(ref) + fp32_err) + fp32_err + TINY[dtype]
