"""ctypes binding of libdora (include/dora.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
layout, their data pointers and the current HIP stream are handed to the C
ABI, and outputs are allocated with torch. Every step of the computation
runs in libdora's kernels; there is no fallback path. If ``libdora.so`` is
missing, every call raises.

The function names match the C entry points.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import NamedTuple

import torch

__all__ = [
    "LIB_PATH",
    "DoraError",
    "load",
    "dora_version",
    "dora_status_string",
    "dora_norm_chunk_size",
    "dora_norm_workspace_size",
    "dora_norm_plan_info",
    "dora_factored_norm",
    "dora_magnitude_scale",
    "dora_norm_to_dtype",
    "dora_layer_output",
    "dora_compose",
    "DORA_BF16",
    "DORA_F32",
    "DORA_F16",
    "PLAN_FIELDS",
    "dora_compose_backward",
    "dora_compose_backward_workspace_size",
    "dora_factored_norm_marked",
    "dora_factored_norm_noalloc",
    "NOALLOC_SCRATCH_BYTES",
    "DORA_E4M3",
    "ACTS",
    "dora_rms_norm",
    "dora_rms_norm_quant",
    "dora_rms_norm_backward",
    "dora_rms_norm_backward_workspace_size",
    "dora_matmul",
    "dora_matmul_workspace_size",
    "dora_matmul_plan_info",
    "dora_matmul_backward",
    "dora_matmul_backward_workspace_size",
    "DORA_I8",
    "Int8Rows",
    "dora_layer_norm",
    "dora_layer_norm_quant",
    "dora_layer_norm_backward",
    "dora_layer_norm_backward_workspace_size",
    "dora_quantize_rows",
    "dora_dequantize_rows",
    "dora_matmul_int8",
    "dora_matmul_int8_workspace_size",
    "dora_matmul_int8_plan_info",
    "dora_matmul_backward_int8",
    "dora_matmul_backward_int8_workspace_size",
    "dora_matmul_backward_int8_plan_info",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdora.so")

DORA_BF16 = 0
DORA_F32 = 1
DORA_F16 = 2
DORA_E4M3 = 3   # 8-bit operands of dora_matmul and 8-bit outputs of the norms
DORA_I8 = 4     # 8-bit integers, where an output's 8-bit type is chosen
DEFAULT_BUDGET = 256 << 20
NOALLOC_SCRATCH_BYTES = 32 << 20   # DORA_NOALLOC_SCRATCH_BYTES

PLAN_FIELDS = (
    "mode", "tile_cols", "col_tiles", "gram_tile_cols", "gram_col_tiles", "fast_cfg", "gen_cfg",
    "gram_fast_cfg", "gram_gen_cfg", "granule", "granules", "w_ranges", "gram_ranges", "workspace_bytes",
    "w_grid", "gram_grid", "lds_bytes", "tile_rows", "gram_folded", "gram_symmetric", "gram_term_fused",
    "w_launch", "offsets32", "dense_row_tiles", "dense_col_tiles", "die_groups",
)

_lib = None
_c_i64 = ctypes.c_int64
_c_sz = ctypes.c_size_t
_c_p = ctypes.c_void_p
_c_f = ctypes.c_float
_c_i = ctypes.c_int


class DoraError(RuntimeError):
    """A libdora call returned a non-zero status."""

    def __init__(self, func: str, status: int):
        self.status = status
        super().__init__(f"{func}: {dora_status_string(status)} (status {status})")


def load():
    """Load libdora.so (after torch, so it binds to torch's HIP runtime)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is not built; run `python -m dora_weight_norm_amd.build` "
            "or __graft_entry__.build()"
        )
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "dora_status_string": (ctypes.c_char_p, [_c_i]),
        "dora_version": (_c_i, []),
        "dora_norm_chunk_size": (_c_i, [_c_i64, _c_i64, _c_sz, ctypes.POINTER(_c_i64)]),
        "dora_norm_workspace_size": (_c_i, [_c_i64, _c_i64, _c_i64, _c_i, _c_f, _c_sz, ctypes.POINTER(_c_sz)]),
        "dora_norm_plan_info": (_c_i, [_c_i64, _c_i64, _c_i64, _c_i, _c_f, _c_sz, ctypes.POINTER(_c_i64), _c_i]),
        "dora_factored_norm": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_i64, _c_i64, _c_i64, _c_f, _c_sz, _c_p, _c_sz,
                                      _c_p, _c_p, _c_f, _c_p, _c_p]),
        "dora_factored_norm_marked": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_i64, _c_i64, _c_i64, _c_f, _c_sz, _c_p,
                                             _c_sz, _c_p, _c_p, _c_f, _c_p, _c_p, ctypes.POINTER(_c_p), _c_i]),
        "dora_factored_norm_noalloc": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_i64, _c_i64, _c_i64, _c_f, _c_sz, _c_p,
                                              _c_p, _c_f, _c_p, _c_p]),
        "dora_magnitude_scale": (_c_i, [_c_p, _c_p, _c_f, _c_i64, _c_p, _c_p]),
        "dora_norm_to_dtype": (_c_i, [_c_p, _c_i64, _c_i, _c_p, _c_p]),
        "dora_compose": (_c_i, [_c_p, _c_p, _c_p, _c_f, _c_i, _c_i64, _c_i64, _c_p, _c_p]),
        "dora_layer_output": (_c_i, [_c_p, _c_p, _c_p, _c_f, _c_i, _c_i64, _c_i64, _c_p, _c_p]),
        "dora_compose_backward_workspace_size": (_c_i, [_c_i64, _c_i64, ctypes.POINTER(_c_sz)]),
        "dora_compose_backward": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_f, _c_i, _c_i64, _c_i64, _c_p, _c_p, _c_p,
                                         _c_p, _c_f, _c_p, _c_p, _c_sz, _c_p]),
        "dora_rms_norm": (_c_i, [_c_p, _c_p, _c_p, _c_f, _c_i, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]),
        "dora_rms_norm_backward_workspace_size": (_c_i, [_c_i64, _c_i64, _c_i, ctypes.POINTER(_c_sz)]),
        "dora_rms_norm_backward": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_i, _c_i64, _c_i64, _c_p, _c_p, _c_p,
                                          _c_sz, _c_p]),
        "dora_matmul_workspace_size": (_c_i, [_c_i64, _c_i64, _c_i64, _c_i64, _c_i, _c_i, ctypes.POINTER(_c_sz)]),
        "dora_matmul_plan_info": (_c_i, [_c_i64, _c_i64, _c_i64, _c_i64, _c_i, _c_i, ctypes.POINTER(_c_i64), _c_i]),
        "dora_matmul": (_c_i, [_c_p, _c_p, _c_i, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_f, _c_p,
                               _c_i, _c_p, _c_i, _c_p, _c_p, _c_p, _c_sz, _c_p]),
        "dora_matmul_backward_workspace_size": (_c_i, [_c_i64, _c_i64, _c_i64, _c_i, _c_i, ctypes.POINTER(_c_sz)]),
        "dora_matmul_backward": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_i, _c_p,
                                        _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
        "dora_matmul_backward_rows": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p,
                                             _c_i, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
        "dora_layer_norm": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_f, _c_i, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_i, _c_p,
                                   _c_p, _c_p, _c_p]),
        "dora_layer_norm_backward_workspace_size": (_c_i, [_c_i64, _c_i64, _c_i, ctypes.POINTER(_c_sz)]),
        "dora_layer_norm_backward": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i, _c_i64, _c_i64, _c_p, _c_p, _c_p,
                                            _c_p, _c_sz, _c_p]),
        "dora_quantize_rows": (_c_i, [_c_p, _c_i, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p]),
        "dora_dequantize_rows": (_c_i, [_c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i, _c_p, _c_p]),
        "dora_matmul_int8_workspace_size": (_c_i, [_c_i64, _c_i64, _c_i64, _c_i64, _c_i, ctypes.POINTER(_c_sz)]),
        "dora_matmul_int8_plan_info": (_c_i, [_c_i64, _c_i64, _c_i64, _c_i64, _c_i, ctypes.POINTER(_c_i64), _c_i]),
        "dora_matmul_int8": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_i64, _c_f,
                                    _c_p, _c_i, _c_p, _c_i, _c_p, _c_p, _c_p, _c_sz, _c_p]),
        "dora_matmul_backward_int8_workspace_size": (_c_i, [_c_i64, _c_i64, _c_i64, _c_i, _c_i, _c_i,
                                                            ctypes.POINTER(_c_sz)]),
        "dora_matmul_backward_int8_scales_workspace_size": (_c_i, [_c_i64, _c_i64, _c_i64, _c_i, _c_i, _c_i64, _c_i64,
                                                                   ctypes.POINTER(_c_sz)]),
        "dora_matmul_backward_int8_plan_info": (_c_i, [_c_i64, _c_i64, _c_i64, _c_i, _c_i, _c_i64, _c_i64,
                                                       ctypes.POINTER(_c_i64), _c_i]),
        "dora_matmul_backward_int8": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i, _c_i64, _c_i64, _c_i64,
                                             _c_p, _c_p, _c_p, _c_i, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _call(name: str, *args) -> None:
    st = getattr(_lib or load(), name)(*args)
    if st != 0:
        raise DoraError(name, st)


def _call_on(dev: int, name: str, *args) -> None:
    """_call with GPU `dev`, the tensors' and the stream's, as the current one."""
    if _current_device() == dev:
        _call(name, *args)
    else:
        with torch.cuda.device(dev):
            _call(name, *args)


def dora_version() -> int:
    return load().dora_version()


def dora_status_string(status: int) -> str:
    return load().dora_status_string(status).decode()


def _dtype_code(dtype) -> int:
    if dtype in (torch.bfloat16, "bf16", DORA_BF16):
        return DORA_BF16
    if dtype in (torch.float32, "f32", DORA_F32):
        return DORA_F32
    if dtype in (torch.float16, "f16", DORA_F16):
        return DORA_F16
    raise TypeError(f"unsupported dtype {dtype}; libdora takes bfloat16, float16 or float32")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")


def _out_like(t, name: str, shape, dtype, device):
    """A caller-supplied output buffer: on `device`, contiguous, exactly
    `shape` and `dtype` (the C ABI cannot see allocation sizes, so a short
    or mistyped buffer is refused here, before any launch)."""
    _dev(t, name)
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _workspace(t, name: str, need: int, device):
    """A caller-supplied workspace: on `device`, contiguous, at least `need` bytes."""
    _dev(t, name)
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.numel() * t.element_size() < need:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes; {need} are needed")


# (the index alone, without the checks around it)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(stream, device=None):
    """Allocations made inside belong to `stream` (torch's caching allocator
    then reuses their memory only after the work queued on `stream`), so
    temporaries freed on return cannot be handed to other work while the
    kernels launched on `stream` still use them. Without a stream, `device`
    (of the tensors) is the current GPU inside: the null stream and the
    library's launches are the current GPU's."""
    if stream is not None:
        return torch.cuda.stream(stream)
    if device is not None and device.index != _current_device():
        return torch.cuda.device(device)
    return contextlib.nullcontext()


def dora_norm_chunk_size(d_out: int, d_in: int, budget_bytes: int = DEFAULT_BUDGET) -> int:
    cs = _c_i64()
    _call("dora_norm_chunk_size", d_out, d_in, budget_bytes, ctypes.byref(cs))
    return cs.value


def dora_norm_workspace_size(d_out: int, d_in: int, r: int, dtype, s: float,
                             budget_bytes: int = DEFAULT_BUDGET) -> int:
    ws = _c_sz()
    _call("dora_norm_workspace_size", d_out, d_in, r, _dtype_code(dtype), s, budget_bytes, ctypes.byref(ws))
    return ws.value


def dora_norm_plan_info(d_out: int, d_in: int, r: int, dtype, s: float,
                        budget_bytes: int = DEFAULT_BUDGET) -> dict:
    buf = (_c_i64 * len(PLAN_FIELDS))()
    _call("dora_norm_plan_info", d_out, d_in, r, _dtype_code(dtype), s, budget_bytes, buf, len(PLAN_FIELDS))
    return dict(zip(PLAN_FIELDS, list(buf)))


def dora_factored_norm(W, A, B, s: float, budget_bytes: int = DEFAULT_BUDGET, m=None, eps: float = 1e-6,
                       workspace=None, wnorm=None, g=None, stream=None, events=None):
    """wnorm = ||W + s B A||_row (fp32) and, if m is given, g = m / max(wnorm, eps).

    W [d_out, d_in], A [r, d_in], B [d_out, r], all of one dtype (bfloat16,
    float16 or float32), on the GPU. Returns (wnorm, g); g is None when m is
    None. `events` (a sequence of recorded torch.cuda.Event objects or None
    entries) selects dora_factored_norm_marked, which records them between
    the call's launches.
    """
    for t, nm in ((W, "W"), (A, "A"), (B, "B")):
        _dev(t, nm)
    if W.dim() != 2 or A.dim() != 2 or B.dim() != 2:
        raise ValueError("W, A, B must be 2-D")
    d_out, d_in = W.shape
    r = A.shape[0]
    if A.shape[1] != d_in or tuple(B.shape) != (d_out, r):
        raise ValueError(f"shape mismatch: W {tuple(W.shape)}, A {tuple(A.shape)}, B {tuple(B.shape)}")
    if not (W.dtype == A.dtype == B.dtype):
        raise TypeError("W, A, B must share one dtype")
    if not (W.device == A.device == B.device):
        raise ValueError("W, A, B must be on one device")
    dt = _dtype_code(W.dtype)
    dev = W.device
    ws_bytes = dora_norm_workspace_size(d_out, d_in, r, dt, s, budget_bytes)
    if workspace is not None:
        _workspace(workspace, "workspace", ws_bytes, dev)
    if wnorm is not None:
        _out_like(wnorm, "wnorm", (d_out,), torch.float32, dev)
    if m is not None:
        _out_like(m, "m", (d_out,), torch.float32, dev)
        if g is not None:
            _out_like(g, "g", (d_out,), torch.float32, dev)
    with _on(stream, dev):
        if workspace is None and ws_bytes > 0:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        if wnorm is None:
            wnorm = torch.empty(d_out, dtype=torch.float32, device=dev)
        if m is not None and g is None:
            g = torch.empty(d_out, dtype=torch.float32, device=dev)
        args = (_ptr(W), _ptr(A), _ptr(B), dt, d_out, d_in, r, s, budget_bytes, _ptr(workspace),
                0 if workspace is None else workspace.numel() * workspace.element_size(),
                _ptr(wnorm), _ptr(m), eps, _ptr(g) if m is not None else None, _stream(stream))
        if events is None:
            _call("dora_factored_norm", *args)
        else:
            handles = [None if e is None else int(getattr(e, "cuda_event", e)) for e in events]
            if any(h == 0 for h in handles):
                raise ValueError("an event has no HIP handle yet (record it once first)")
            arr = (_c_p * max(len(handles), 1))(*handles)
            _call("dora_factored_norm_marked", *args, arr, len(handles))
    return wnorm, (g if m is not None else None)


def dora_factored_norm_marked(W, A, B, s: float, events, **kw):
    """dora_factored_norm with HIP events recorded between its launches
    (events[0] before the first, events[i] after the i-th; None entries
    skipped). Same keywords and results as dora_factored_norm."""
    return dora_factored_norm(W, A, B, s, events=list(events), **kw)


def dora_factored_norm_noalloc(W, A, B, s: float, budget_bytes: int = DEFAULT_BUDGET, m=None, eps: float = 1e-6,
                               wnorm=None, g=None, stream=None):
    """dora_factored_norm with the library's per-GPU scratch array as its
    workspace (the C call allocates nothing). wnorm and g may be passed in,
    so that the call itself allocates nothing either. Returns (wnorm, g)."""
    for t, nm in ((W, "W"), (A, "A"), (B, "B")):
        _dev(t, nm)
    if W.dim() != 2 or A.dim() != 2 or B.dim() != 2:
        raise ValueError("W, A, B must be 2-D")
    d_out, d_in = W.shape
    r = A.shape[0]
    if A.shape[1] != d_in or tuple(B.shape) != (d_out, r):
        raise ValueError(f"shape mismatch: W {tuple(W.shape)}, A {tuple(A.shape)}, B {tuple(B.shape)}")
    if not (W.dtype == A.dtype == B.dtype):
        raise TypeError("W, A, B must share one dtype")
    if not (W.device == A.device == B.device):
        raise ValueError("W, A, B must be on one device")
    dev = W.device
    if wnorm is not None:
        _out_like(wnorm, "wnorm", (d_out,), torch.float32, dev)
    if m is not None:
        _out_like(m, "m", (d_out,), torch.float32, dev)
        if g is not None:
            _out_like(g, "g", (d_out,), torch.float32, dev)
    with _on(stream, dev):
        if wnorm is None:
            wnorm = torch.empty(d_out, dtype=torch.float32, device=dev)
        if m is not None and g is None:
            g = torch.empty(d_out, dtype=torch.float32, device=dev)
        _call("dora_factored_norm_noalloc", _ptr(W), _ptr(A), _ptr(B), _dtype_code(W.dtype), d_out, d_in, r, s,
              budget_bytes, _ptr(wnorm), _ptr(m), eps, _ptr(g) if m is not None else None, _stream(stream))
    return wnorm, (g if m is not None else None)


def dora_magnitude_scale(m, wnorm, eps: float = 1e-6, g=None, stream=None):
    """g = m / max(wnorm, eps), fp32 [d_out]."""
    _dev(m, "m")
    if m.dtype != torch.float32 or m.dim() != 1:
        raise ValueError("m must be float32 [d_out]")
    _out_like(wnorm, "wnorm", m.shape, torch.float32, m.device)
    if g is not None:
        _out_like(g, "g", m.shape, torch.float32, m.device)
    with _on(stream, m.device):
        if g is None:
            g = torch.empty_like(m)
        _call("dora_magnitude_scale", _ptr(m), _ptr(wnorm), eps, m.numel(), _ptr(g), _stream(stream))
    return g


def dora_norm_to_dtype(wnorm, dtype, out=None, stream=None):
    """wnorm (fp32 [n]) rounded to `dtype` (bfloat16, float16 or float32), nearest even."""
    _dev(wnorm, "wnorm")
    if wnorm.dtype != torch.float32 or wnorm.dim() != 1:
        raise ValueError("wnorm must be float32 [n]")
    tdt = {DORA_BF16: torch.bfloat16, DORA_F32: torch.float32, DORA_F16: torch.float16}[_dtype_code(dtype)]
    if out is not None:
        _out_like(out, "out", wnorm.shape, tdt, wnorm.device)
    with _on(stream, wnorm.device):
        if out is None:
            out = torch.empty(wnorm.shape, dtype=tdt, device=wnorm.device)
        _call("dora_norm_to_dtype", _ptr(wnorm), wnorm.numel(), _dtype_code(dtype), _ptr(out), _stream(stream))
    return out


def _compose_call(name, base, lora, g, s, out, stream):
    for t, nm in ((base, "base"), (lora, "lora"), (g, "g")):
        _dev(t, nm)
    if base.shape != lora.shape or base.dtype != lora.dtype:
        raise ValueError("base and lora must share shape and dtype")
    if base.dim() != 2:
        raise ValueError("base and lora must be [T, d_out]")
    T, d_out = base.shape
    if g.dtype != torch.float32 or g.shape != (d_out,):
        raise ValueError("g must be float32 [d_out]")
    if not (base.device == lora.device == g.device):
        raise ValueError("base, lora and g must be on one device")
    dt = _dtype_code(base.dtype)
    if out is not None:
        _out_like(out, "out", base.shape, base.dtype, base.device)
    with _on(stream, base.device):
        if out is None:
            out = torch.empty_like(base)
        _call(name, _ptr(base), _ptr(lora), _ptr(g), s, dt, T, d_out, _ptr(out), _stream(stream))
    return out


def dora_compose(base, lora, g, s: float, out=None, stream=None):
    """out = (g - 1) * base + g * (s * lora), with g [d_out] scaling columns of [T, d_out]."""
    return _compose_call("dora_compose", base, lora, g, s, out, stream)


def dora_layer_output(base, lora, g, s: float, y=None, stream=None):
    """y = base + ((g - 1) * base + g * (s * lora)): the DoRA layer output, one rounding."""
    return _compose_call("dora_layer_output", base, lora, g, s, y, stream)

def dora_compose_backward_workspace_size(T: int, d_out: int) -> int:
    ws = _c_sz()
    _call("dora_compose_backward_workspace_size", T, d_out, ctypes.byref(ws))
    return ws.value


def dora_compose_backward(dy, base, lora, g, s: float, need_dg: bool = True, wnorm=None, eps: float = 1e-6,
                          d_base=None, d_lora=None, workspace=None, stream=None):
    """Gradients of delta = (g - 1) * base + g * (s * lora), the row norm detached.

    Returns (d_base, d_lora, dg, dm): d_base and d_lora like dy; dg fp32
    [d_out] (None when need_dg is False: the magnitude is frozen, base and
    lora are then not read and may be None); dm = dg / max(wnorm, eps) when
    wnorm is given.
    """
    _dev(dy, "dy")
    _dev(g, "g")
    if dy.dim() != 2:
        raise ValueError("dy must be [T, d_out]")
    T, d_out = dy.shape
    if g.dtype != torch.float32 or g.shape != (d_out,):
        raise ValueError("g must be float32 [d_out]")
    if need_dg:
        for t, nm in ((base, "base"), (lora, "lora")):
            _dev(t, nm)
            if t.shape != dy.shape or t.dtype != dy.dtype:
                raise ValueError(f"{nm} must match dy")
    if wnorm is not None:
        if not need_dg:
            raise ValueError("dm needs dg")
        _dev(wnorm, "wnorm")
        if wnorm.dtype != torch.float32 or wnorm.shape != (d_out,):
            raise ValueError("wnorm must be float32 [d_out]")
    dt = _dtype_code(dy.dtype)
    dev = dy.device
    if g.device != dev:
        raise ValueError("g must be on dy's device")
    if d_base is not None:
        _out_like(d_base, "d_base", dy.shape, dy.dtype, dev)
    if d_lora is not None:
        _out_like(d_lora, "d_lora", dy.shape, dy.dtype, dev)
    ws_bytes = dora_compose_backward_workspace_size(T, d_out) if need_dg else 0
    if workspace is not None and ws_bytes > 0:
        _workspace(workspace, "workspace", ws_bytes, dev)
    with _on(stream, dev):
        d_base = torch.empty_like(dy) if d_base is None else d_base
        d_lora = torch.empty_like(dy) if d_lora is None else d_lora
        dg = torch.empty(d_out, dtype=torch.float32, device=dev) if need_dg else None
        dm = torch.empty(d_out, dtype=torch.float32, device=dev) if wnorm is not None else None
        if workspace is None and ws_bytes > 0:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        _call("dora_compose_backward", _ptr(dy), _ptr(base if need_dg else None), _ptr(lora if need_dg else None),
              _ptr(g), s, dt, T, d_out, _ptr(d_base), _ptr(d_lora), _ptr(dg), _ptr(wnorm), eps, _ptr(dm),
              _ptr(workspace), ws_bytes if workspace is not None else 0, _stream(stream))
    return d_base, d_lora, dg, dm


# ---------------------------------------------------------------------------
# The block around the adapted layer: residual RMS norm and matrix product.
# ---------------------------------------------------------------------------
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_TORCH_DT = {torch.bfloat16: DORA_BF16, torch.float32: DORA_F32, torch.float16: DORA_F16}
_E4M3 = torch.float8_e4m3fn
# (the handle alone, without a Stream object around it)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


# A call of a single token takes the GPU a few microseconds, so the checks below
# cost as little as they can: one pass of plain comparisons a tensor, the
# device as its index, and messages only where a check fails.
def _refuse(t, name: str, shape, dtype, dev: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    raise ValueError(f"{name} must be contiguous {dtype} {tuple(shape)} on cuda:{dev}, got {t.dtype} "
                     f"{tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")


def _want(t, name: str, shape, dtype, dev: int) -> int:
    """The address of a contiguous tensor of exactly this shape, dtype and GPU (a host tensor's index is -1)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, shape, dtype, dev)


def _maybe(t, name: str, shape, dtype, dev: int):
    return None if t is None else _want(t, name, shape, dtype, dev)


def _first(t, name: str) -> int:
    """The GPU of the 2-D tensor that a call takes its shapes and dtype from."""
    try:
        dev = t.get_device()
        if dev >= 0 and t.dim() == 2 and t.is_contiguous():
            return dev
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    raise ValueError(f"{name} must be contiguous and 2-D, got {tuple(t.shape)}")


def _type_code(dtype) -> int:
    code = _TORCH_DT.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}; libdora takes bfloat16, float16 or float32")
    return code


def _raw_stream(stream, dev: int) -> int:
    if stream is None:
        return _current_raw_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{dev}")
    return stream.cuda_stream


def _new(stream, shape, dtype, dev: int):
    """A tensor that belongs to `stream` (see _on)."""
    if stream is None:   # (with its strides named it costs 1.3 us of the host's time, 1.7 without)
        strides = (shape[1], 1) if len(shape) == 2 else (1,)
        return torch.empty_strided(shape, strides, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _out(t, name: str, shape, dtype, dev: int, stream):
    """An output and its address: the caller's buffer, checked, or a new one."""
    if t is None:
        t = _new(stream, shape, dtype, dev)
        return t, t.data_ptr()
    return t, _want(t, name, shape, dtype, dev)


def _space(workspace, need: int, stream, dev: int):
    """The caller's workspace, checked, or a new one; None where none is needed."""
    if workspace is not None:
        _workspace(workspace, "workspace", need, torch.device("cuda", dev))
        return workspace
    return _new(stream, (need,), torch.uint8, dev) if need > 0 else None


def _addr(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=4096)
def _size_of(name: str, *args) -> int:
    """A workspace query; a pure function of its arguments."""
    ws = _c_sz()
    _call(name, *args, ctypes.byref(ws))
    return ws.value


def dora_rms_norm_backward_workspace_size(T: int, d: int, dtype) -> int:
    return _size_of("dora_rms_norm_backward_workspace_size", T, d, _dtype_code(dtype))


def _operand_code(dtype) -> int:
    return DORA_E4M3 if dtype in (_E4M3, "e4m3", DORA_E4M3) else _dtype_code(dtype)


def dora_matmul_workspace_size(M: int, N: int, K: int, r: int, dtype, aligned_operands: int = 15) -> int:
    return _size_of("dora_matmul_workspace_size", M, N, K, r, _operand_code(dtype), aligned_operands)


def dora_matmul_plan_info(M: int, N: int, K: int, r: int, dtype, aligned_operands: int = 15) -> dict:
    buf = (_c_i64 * 5)()
    _call("dora_matmul_plan_info", M, N, K, r, _operand_code(dtype), aligned_operands, buf, 5)
    return dict(zip(("tile_rows", "splits", "copies", "workspace_bytes", "few_rows"), list(buf)))


def dora_matmul_backward_workspace_size(M: int, N: int, K: int, dtype, outputs: int = 31) -> int:
    """`outputs`: the sum of the GRAD_ constants that apply."""
    return _size_of("dora_matmul_backward_workspace_size", M, N, K, _dtype_code(dtype), outputs)


def _rms_norm(x, weight, eps, residual, h, rstd, want_rstd, stream, y=None, q=None, scale=None, quant=False):
    dev, dtype, shape = _first(x, "x"), x.dtype, x.shape
    code = _type_code(dtype)
    T, d = shape
    f32 = torch.float32
    pw = pres = ph = prs = py = pq = ps = None
    if weight is not None:
        pw = _want(weight, "weight", (d,), f32, dev)
    if residual is not None:
        pres = _want(residual, "residual", shape, dtype, dev)
        if h is None:
            h = _new(stream, shape, dtype, dev)
        ph = _want(h, "h", shape, dtype, dev)
    elif h is not None:
        raise ValueError("h needs a residual (without one, h is x)")
    if rstd is None and want_rstd:
        rstd = _new(stream, (T,), f32, dev)
    if rstd is not None:
        prs = _want(rstd, "rstd", (T,), f32, dev)
    if quant:
        q = _new(stream, shape, _E4M3, dev) if q is None else q
        scale = _new(stream, (T,), f32, dev) if scale is None else scale
        pq, ps = _want(q, "q", shape, _E4M3, dev), _want(scale, "scale", (T,), f32, dev)
    else:
        y = _new(stream, shape, dtype, dev) if y is None else y
        py = _want(y, "y", shape, dtype, dev)
    _call_on(dev, "dora_rms_norm", x.data_ptr(), pres, pw, eps, code, T, d, ph, py, pq, ps, prs,
             _raw_stream(stream, dev))
    return y, q, scale, (x if residual is None else h), rstd


def dora_rms_norm(x, weight, eps: float, residual=None, y=None, h=None, rstd=None, want_rstd: bool = True,
                  stream=None):
    """y = h * rstd * weight with h = x + residual and rstd = 1 / sqrt(mean h^2 + eps) over each row.

    x, residual [T, d] of one dtype (bfloat16, float16 or float32), weight
    float32 [d] or None. Returns (y, h, rstd): h is x itself without a
    residual; rstd float32 [T] (None with want_rstd False).
    """
    y, _, _, h, rstd = _rms_norm(x, weight, eps, residual, h, rstd, want_rstd, stream, y=y)
    return y, h, rstd


def dora_rms_norm_quant(x, weight, eps: float, residual=None, q=None, scale=None, h=None, rstd=None,
                        want_rstd: bool = True, stream=None):
    """dora_rms_norm with its output in 8 bits: q float8_e4m3fn [T, d] and scale
    float32 [T], the row's largest |value| / 448. Returns (q, scale, h, rstd)."""
    _, q, scale, h, rstd = _rms_norm(x, weight, eps, residual, h, rstd, want_rstd, stream, q=q, scale=scale,
                                     quant=True)
    return q, scale, h, rstd


def dora_rms_norm_backward(dy, h, rstd, weight, dh=None, need_dweight: bool = True, dx=None, dweight=None,
                           workspace=None, stream=None):
    """Gradients of dora_rms_norm from its h and rstd. Returns (dx, dweight):
    dx is the gradient of x and of the residual, dh (optional) what reaches h
    directly is added to it; dweight float32 [d], None if not needed."""
    dev, dtype, shape = _first(dy, "dy"), dy.dtype, dy.shape
    code = _type_code(dtype)
    T, d = shape
    f32 = torch.float32
    ph, prs = _want(h, "h", shape, dtype, dev), _want(rstd, "rstd", (T,), f32, dev)
    pw, pdh = _maybe(weight, "weight", (d,), f32, dev), _maybe(dh, "dh", shape, dtype, dev)
    if dweight is not None and not need_dweight:
        raise ValueError("dweight given but need_dweight is False")
    need = dora_rms_norm_backward_workspace_size(T, d, code) if need_dweight else 0
    dx = _new(stream, shape, dtype, dev) if dx is None else dx
    if need_dweight and dweight is None:
        dweight = _new(stream, (d,), f32, dev)
    pdx, pdw = _want(dx, "dx", shape, dtype, dev), _maybe(dweight, "dweight", (d,), f32, dev)
    workspace = _space(workspace, need, stream, dev)
    _call_on(dev, "dora_rms_norm_backward", dy.data_ptr(), pdh, ph, prs, pw, code, T, d, pdx, pdw, _addr(workspace),
             need, _raw_stream(stream, dev))
    return dx, dweight


def _act(act) -> int:
    if act not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}, got {act!r}")
    return ACTS[act]


def dora_matmul(x, w, row_scale=None, col_scale=None, t=None, b=None, s: float = 1.0, bias=None, act: str = "none",
                residual=None, out_dtype=None, save: bool = False, y=None, u=None, workspace=None, stream=None):
    """y = act(col_scale * u + bias) + residual with u = row_scale * (x w^T + s * t b^T).

    x [M, K] and w [N, K] of one dtype (bfloat16, float16, float32 or
    float8_e4m3fn); t [M, r] and b [N, r] of the same dtype, both or neither
    (neither with float8); row_scale float32 [M]; col_scale, bias float32 [N];
    residual [M, N] of the output's dtype. out_dtype is x's, and for float8
    one of the other three (default bfloat16). act: none, relu, gelu,
    gelu_tanh or silu. Returns (y, u); u, the product that the backward
    takes, is None unless `save` (or a buffer for it) is given. A row_scale
    that the product had goes to the backward too.
    """
    dev, dtype = _first(x, "x"), x.dtype
    e8 = dtype is _E4M3
    code = DORA_E4M3 if e8 else _TORCH_DT.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}; libdora takes bfloat16, float16, float32 or float8_e4m3fn")
    M, K = x.shape
    _first(w, "w")
    N = w.shape[0]
    px, pw = x.data_ptr(), _want(w, "w", (N, K), dtype, dev)
    odt = out_dtype if out_dtype is not None else (torch.bfloat16 if e8 else dtype)
    out_code = _TORCH_DT.get(odt)
    if out_code is None or (not e8 and odt is not dtype):
        raise TypeError(f"out_dtype {odt} does not go with {dtype}")
    r, pt, pb = 0, None, None
    al = ((px & 15) == 0) | ((pw & 15) == 0) << 1
    if t is not None or b is not None:
        if t is None or b is None:
            raise ValueError("t and b come together")
        if e8:
            raise TypeError("a low-rank pair does not go with float8 operands")
        _first(t, "t")
        r = t.shape[1]
        pt, pb = _want(t, "t", (M, r), dtype, dev), _want(b, "b", (N, r), dtype, dev)
        al |= ((pt & 15) == 0) << 2 | ((pb & 15) == 0) << 3
    f32, out = torch.float32, (M, N)
    prow = _maybe(row_scale, "row_scale", (M,), f32, dev)
    pcol, pbias = _maybe(col_scale, "col_scale", (N,), f32, dev), _maybe(bias, "bias", (N,), f32, dev)
    pres = _maybe(residual, "residual", out, odt, dev)
    act_code = _act(act)
    need = _size_of("dora_matmul_workspace_size", M, N, K, r, code, al)
    y = _new(stream, out, odt, dev) if y is None else y
    if u is None and save:
        u = _new(stream, out, odt, dev)
    py, pu = _want(y, "y", out, odt, dev), _maybe(u, "u", out, odt, dev)
    workspace = _space(workspace, need, stream, dev)
    _call_on(dev, "dora_matmul", px, pw, code, M, N, K, prow, pcol, pt, pb, r, s, pbias, act_code, pres, out_code, py,
             pu, _addr(workspace), need, _raw_stream(stream, dev))
    return y, u


GRAD_DX, GRAD_DW, GRAD_SUMS, GRAD_DU, GRAD_ALIGNED = 1, 2, 4, 8, 16   # DORA_GRAD_*


def dora_matmul_backward(dy, u, x, w, col_scale=None, bias=None, act: str = "none", need_dx: bool = True,
                         need_dw: bool = True, need_dbias: bool = True, need_dcol_scale: bool = True,
                         workspace=None, stream=None, row_scale=None):
    """Gradients of dora_matmul from its u (bfloat16, float16 or float32),
    with the row_scale, col_scale, bias and act that it had.

    Returns (dx, dw, dbias, dcol_scale, du): dx [M, K], dw [N, K], dbias and
    dcol_scale float32 [N] (each None if not needed), and du [M, N], the
    gradient of x w^T + s * t b^T (of u, where there is no row_scale). x is
    read for dw and w for dx; either may be None where its product is not
    needed. The residual's gradient is dy; row_scale's is not computed.
    """
    dev, dtype = _first(dy, "dy"), dy.dtype
    code = _type_code(dtype)
    M, N = out = dy.shape
    pu = _want(u, "u", out, dtype, dev)
    if need_dx and w is None or need_dw and x is None:
        raise ValueError("dx needs w, and dw needs x")
    K = 0
    if x is not None:
        _first(x, "x")
        K = x.shape[1]
        _want(x, "x", (M, K), dtype, dev)
    if w is not None:
        _first(w, "w")
        K = w.shape[1] if x is None else K
        _want(w, "w", (N, K), dtype, dev)
    f32 = torch.float32
    pcol, pbias = _maybe(col_scale, "col_scale", (N,), f32, dev), _maybe(bias, "bias", (N,), f32, dev)
    prow = _maybe(row_scale, "row_scale", (M,), f32, dev)
    act_code = _act(act)
    du = _new(stream, out, dtype, dev)
    dx = _new(stream, (M, K), dtype, dev) if need_dx else None
    dw = _new(stream, (N, K), dtype, dev) if need_dw else None
    dbias = _new(stream, (N,), f32, dev) if need_dbias else None
    dcol = _new(stream, (N,), f32, dev) if need_dcol_scale else None
    outputs = (GRAD_DX * need_dx + GRAD_DW * need_dw + GRAD_SUMS * (need_dbias or need_dcol_scale)
               + GRAD_DU * (du.data_ptr() % 16 == 0)
               + GRAD_ALIGNED * ((not need_dw or x.data_ptr() % 16 == 0) and (not need_dx or w.data_ptr() % 16 == 0)))
    need = _size_of("dora_matmul_backward_workspace_size", M, N, K, code, outputs)
    workspace = _space(workspace, need, stream, dev)
    _call_on(dev, "dora_matmul_backward_rows", dy.data_ptr(), pu, _addr(x) if need_dw else None,
             _addr(w) if need_dx else None, code, M, N, K, prow, pcol, pbias, act_code, _addr(du), _addr(dx),
             _addr(dw), _addr(dbias), _addr(dcol), _addr(workspace), need, _raw_stream(stream, dev))
    return dx, dw, dbias, dcol, du


# ---------------------------------------------------------------------------
# Rows held in 8-bit integers: the layer norm that writes them, packing, the
# integer product, and the backward that reads them as checkpoints.
# ---------------------------------------------------------------------------
class Int8Rows(NamedTuple):
    """Rows in 8-bit integers: q int8 [T, d]; scale float32 [T] with group 0, else [T, ceil(d / group)]."""
    q: torch.Tensor
    scale: torch.Tensor
    group: int = 0


class _Int8RowsArg(ctypes.Structure):
    _fields_ = [("q", _c_p), ("scale", _c_p), ("group", _c_i64)]


_Q8_CODE = {torch.int8: DORA_I8, _E4M3: DORA_E4M3}
GROUPS = (0, 32, 64, 128, 256)
HELD_X, HELD_W = 1, 2   # DORA_HELD_*


def _scale_shape(T: int, d: int, group: int) -> tuple:
    if group not in GROUPS:
        raise ValueError(f"group must be one of {GROUPS}, got {group!r}")
    return (T, -(-d // group)) if group else (T,)


def dora_layer_norm_backward_workspace_size(T: int, d: int, dtype) -> int:
    return _size_of("dora_layer_norm_backward_workspace_size", T, d, _dtype_code(dtype))


def dora_matmul_int8_workspace_size(M: int, N: int, K: int, r: int, aligned_operands: int = 15) -> int:
    return _size_of("dora_matmul_int8_workspace_size", M, N, K, r, aligned_operands)


INT8_KERNELS = ("tiles", "few_rows", "walk", "tiles_anywhere")
HELD_READS = ("as_given", "copy", "int8_rows")


def dora_matmul_int8_plan_info(M: int, N: int, K: int, r: int, aligned_operands: int = 15) -> dict:
    """`kernel`: one of INT8_KERNELS, or None where there is nothing to do."""
    buf = (_c_i64 * 6)()
    _call("dora_matmul_int8_plan_info", M, N, K, r, aligned_operands, buf, 6)
    info = dict(zip(("tile_rows", "splits", "copies", "workspace_bytes", "few_rows"), list(buf)))
    info["kernel"] = None if buf[5] < 0 else INT8_KERNELS[buf[5]]
    return info


def dora_matmul_backward_int8_workspace_size(M: int, N: int, K: int, dtype, outputs: int = 31, held: int = 3) -> int:
    """`outputs`: the sum of the GRAD_ constants that apply; `held`: of the HELD_ ones."""
    return _size_of("dora_matmul_backward_int8_workspace_size", M, N, K, _dtype_code(dtype), outputs, held)


def dora_matmul_backward_int8_plan_info(M: int, N: int, K: int, dtype, outputs: int = 31, x_scales: int = 1,
                                        w_scales: int = 1) -> dict:
    """For dx and dw (None where there is none) the product's tile_rows, its splits, and how it `reads` w or x (one of
    HELD_READS), and workspace_bytes. `outputs`: the sum of the GRAD_ constants that apply; `x_scales`, `w_scales`: how
    many scales a row of x and w has, 0 where they are not Int8Rows."""
    buf = (_c_i64 * 7)()
    _call("dora_matmul_backward_int8_plan_info", M, N, K, _dtype_code(dtype), outputs, x_scales, w_scales, buf, 7)
    info = {"workspace_bytes": buf[6]}
    for name, at in (("dx", 0), ("dw", 3)):
        info[name] = None if buf[at] < 0 else {"tile_rows": buf[at], "splits": buf[at + 1],
                                               "reads": HELD_READS[buf[at + 2]]}
    return info


def _layer_norm(x, weight, bias, eps, residual, h, mean, rstd, want_stats, stream, y=None, q=None, scale=None,
                q_dtype=None, want_y=True):
    dev, dtype, shape = _first(x, "x"), x.dtype, x.shape
    code = _type_code(dtype)
    T, d = shape
    f32 = torch.float32
    ph = py = pq = ps = None
    pw, pb = _maybe(weight, "weight", (d,), f32, dev), _maybe(bias, "bias", (d,), f32, dev)
    pres = _maybe(residual, "residual", shape, dtype, dev)
    if residual is not None:
        h, ph = _out(h, "h", shape, dtype, dev, stream)
    elif h is not None:
        raise ValueError("h needs a residual (without one, h is x)")
    if want_stats:
        mean, pm = _out(mean, "mean", (T,), f32, dev, stream)
        rstd, prs = _out(rstd, "rstd", (T,), f32, dev, stream)
    else:
        pm, prs = _maybe(mean, "mean", (T,), f32, dev), _maybe(rstd, "rstd", (T,), f32, dev)
    if q_dtype is not None:
        q, pq = _out(q, "q", shape, q_dtype, dev, stream)
        scale, ps = _out(scale, "scale", (T,), f32, dev, stream)
    if want_y or y is not None:
        y, py = _out(y, "y", shape, dtype, dev, stream)
    _call_on(dev, "dora_layer_norm", x.data_ptr(), pres, pw, pb, eps, code, T, d, ph, py, pq, _Q8_CODE.get(q_dtype, 0),
             ps, pm, prs, _raw_stream(stream, dev))
    return y, q, scale, (x if residual is None else h), mean, rstd


def dora_layer_norm(x, weight, bias, eps: float, residual=None, y=None, h=None, mean=None, rstd=None,
                    want_stats: bool = True, stream=None):
    """y = (h - mean) * rstd * weight + bias with h = x + residual, over each row.

    x, residual [T, d] of one dtype (bfloat16, float16 or float32), weight and
    bias float32 [d] or None. Returns (y, h, mean, rstd): h is x itself without
    a residual; mean and rstd float32 [T] (None with want_stats False).
    """
    y, _, _, h, mean, rstd = _layer_norm(x, weight, bias, eps, residual, h, mean, rstd, want_stats, stream, y=y)
    return y, h, mean, rstd


def dora_layer_norm_quant(x, weight, bias, eps: float, q_dtype=torch.int8, residual=None, q=None, scale=None, h=None,
                          mean=None, rstd=None, want_stats: bool = True, y=None, stream=None):
    """dora_layer_norm with its output in 8 bits: q [T, d] of q_dtype (int8 or
    float8_e4m3fn) and scale float32 [T], the row's largest |value| / 127 or / 448.
    Returns (q, scale, h, mean, rstd). y, if a buffer for it is given, receives
    the output in x's dtype as well."""
    if q_dtype not in _Q8_CODE:   # (None too, which would leave q as it was)
        raise TypeError(f"q_dtype must be int8 or float8_e4m3fn, got {q_dtype}")
    _, q, scale, h, mean, rstd = _layer_norm(x, weight, bias, eps, residual, h, mean, rstd, want_stats, stream, y=y,
                                             q=q, scale=scale, q_dtype=q_dtype, want_y=False)
    return q, scale, h, mean, rstd


def dora_layer_norm_backward(dy, h, mean, rstd, weight, dh=None, need_dweight: bool = True, need_dbias: bool = True,
                             dx=None, dweight=None, dbias=None, workspace=None, stream=None):
    """Gradients of dora_layer_norm from its h, mean and rstd. Returns (dx,
    dweight, dbias): dx is the gradient of x and of the residual, dh (optional)
    what reaches h directly is added to it; dweight and dbias float32 [d], None
    where not needed."""
    dev, dtype, shape = _first(dy, "dy"), dy.dtype, dy.shape
    code = _type_code(dtype)
    T, d = shape
    f32 = torch.float32
    ph = _want(h, "h", shape, dtype, dev)
    pm, prs = _want(mean, "mean", (T,), f32, dev), _want(rstd, "rstd", (T,), f32, dev)
    pw, pdh = _maybe(weight, "weight", (d,), f32, dev), _maybe(dh, "dh", shape, dtype, dev)
    if dweight is not None and not need_dweight or dbias is not None and not need_dbias:
        raise ValueError("a gradient's buffer is given but the gradient is not needed")
    need = dora_layer_norm_backward_workspace_size(T, d, code) if need_dweight or need_dbias else 0
    dx, pdx = _out(dx, "dx", shape, dtype, dev, stream)
    pdw = pdb = None
    if need_dweight:
        dweight, pdw = _out(dweight, "dweight", (d,), f32, dev, stream)
    if need_dbias:
        dbias, pdb = _out(dbias, "dbias", (d,), f32, dev, stream)
    workspace = _space(workspace, need, stream, dev)
    _call_on(dev, "dora_layer_norm_backward", dy.data_ptr(), pdh, ph, pm, prs, pw, code, T, d, pdx, pdw, pdb,
             _addr(workspace), need, _raw_stream(stream, dev))
    return dx, dweight, dbias


def dora_quantize_rows(x, group: int = 0, q=None, scale=None, stream=None):
    """x [T, d] as int8 rows: (q int8 [T, d], scale float32), scale = max |x| / 127
    over a row ([T], group 0) or over each group of 32, 64, 128 or 256 columns of
    it ([T, ceil(d / group)]), and q = x / scale to the nearest integer."""
    dev, shape = _first(x, "x"), x.shape
    code = _type_code(x.dtype)
    T, d = shape
    scales = _scale_shape(T, d, group)
    q, pq = _out(q, "q", shape, torch.int8, dev, stream)
    scale, ps = _out(scale, "scale", scales, torch.float32, dev, stream)
    _call_on(dev, "dora_quantize_rows", x.data_ptr(), code, T, d, group, pq, ps, _raw_stream(stream, dev))
    return q, scale


def dora_dequantize_rows(q, scale, group: int = 0, dtype=torch.bfloat16, out=None, stream=None):
    """The values q * scale that int8 rows stand for, [T, d] rounded once to `dtype` (bfloat16, float16 or float32)."""
    dev, shape = _first(q, "q"), q.shape
    T, d = shape
    pq = _want(q, "q", shape, torch.int8, dev)
    ps = _want(scale, "scale", _scale_shape(T, d, group), torch.float32, dev)
    code = _type_code(dtype)
    out, po = _out(out, "out", shape, dtype, dev, stream)
    _call_on(dev, "dora_dequantize_rows", pq, ps, T, d, group, code, po, _raw_stream(stream, dev))
    return out


def dora_matmul_int8(x, w, row_scale, w_scale, col_scale=None, t=None, b=None, s: float = 1.0, bias=None,
                     act: str = "none", residual=None, out_dtype=torch.bfloat16, save: bool = False, y=None, u=None,
                     workspace=None, stream=None):
    """y = act(col_scale * u + bias) + residual with u = row_scale * w_scale * (x w^T) + s * t b^T.

    x int8 [M, K] with row_scale float32 [M] and w int8 [N, K] with w_scale
    float32 [N] are int8 rows with one scale a row; t [M, r] and b [N, r] of
    out_dtype, both or neither (neither with float32); col_scale, bias float32
    [N]; residual [M, N] of out_dtype. Returns (y, u); u, the product that the
    backward takes, is None unless `save` (or a buffer for it) is given.
    """
    dev = _first(x, "x")
    M, K = x.shape
    _first(w, "w")
    N = w.shape[0]
    i8, f32 = torch.int8, torch.float32
    px, pw = _want(x, "x", (M, K), i8, dev), _want(w, "w", (N, K), i8, dev)
    prow, pws = _want(row_scale, "row_scale", (M,), f32, dev), _want(w_scale, "w_scale", (N,), f32, dev)
    out_code = _type_code(out_dtype)
    r, pt, pb = 0, None, None
    al = ((px & 15) == 0) | ((pw & 15) == 0) << 1
    if t is not None or b is not None:
        if t is None or b is None:
            raise ValueError("t and b come together")
        if out_dtype is f32:
            raise TypeError("a low-rank pair does not go with float32 outputs of the integer product")
        _first(t, "t")
        r = t.shape[1]
        pt, pb = _want(t, "t", (M, r), out_dtype, dev), _want(b, "b", (N, r), out_dtype, dev)
        al |= ((pt & 15) == 0) << 2 | ((pb & 15) == 0) << 3
    out = (M, N)
    pcol, pbias = _maybe(col_scale, "col_scale", (N,), f32, dev), _maybe(bias, "bias", (N,), f32, dev)
    pres = _maybe(residual, "residual", out, out_dtype, dev)
    act_code = _act(act)
    need = _size_of("dora_matmul_int8_workspace_size", M, N, K, r, al)
    y, py = _out(y, "y", out, out_dtype, dev, stream)
    pu = None
    if save or u is not None:
        u, pu = _out(u, "u", out, out_dtype, dev, stream)
    workspace = _space(workspace, need, stream, dev)
    _call_on(dev, "dora_matmul_int8", px, prow, pw, pws, M, N, K, pcol, pt, pb, r, s, pbias, act_code, pres, out_code,
             py, pu, _addr(workspace), need, _raw_stream(stream, dev))
    return y, u


def _held(v, name: str, shape, dtype, dev: int):
    """(address, structure) of an operand in the storage type or as Int8Rows; the other one is None."""
    if not isinstance(v, Int8Rows):
        return _want(v, name, shape, dtype, dev), None
    pq = _want(v.q, f"{name}.q", shape, torch.int8, dev)
    ps = _want(v.scale, f"{name}.scale", _scale_shape(*shape, v.group), torch.float32, dev)
    return None, _Int8RowsArg(pq, ps, v.group)


def dora_matmul_backward_int8(dy, u, x, w, col_scale=None, bias=None, act: str = "none", need_dx: bool = True,
                              need_dw: bool = True, need_dbias: bool = True, need_dcol_scale: bool = True,
                              workspace=None, stream=None, row_scale=None):
    """dora_matmul_backward with any of u, x and w given as Int8Rows.

    u and x are activations packed in the forward (dora_quantize_rows), w a
    frozen 8-bit base. u's values are taken in fp32, x's and w's as operands of
    dy's dtype. Arguments and results otherwise as there: (dx, dw, dbias,
    dcol_scale, du).
    """
    dev, dtype = _first(dy, "dy"), dy.dtype
    code = _type_code(dtype)
    M, N = out = dy.shape
    if need_dx and w is None or need_dw and x is None:
        raise ValueError("dx needs w, and dw needs x")
    K = 0
    for v, name in ((w, "w"), (x, "x")):
        if v is not None:
            v = v.q if isinstance(v, Int8Rows) else v
            _first(v, name)
            K = v.shape[1]
    pu, u8 = _held(u, "u", out, dtype, dev)
    px, x8 = (None, None) if x is None else _held(x, "x", (M, K), dtype, dev)
    pw, w8 = (None, None) if w is None else _held(w, "w", (N, K), dtype, dev)
    f32 = torch.float32
    pcol, pbias = _maybe(col_scale, "col_scale", (N,), f32, dev), _maybe(bias, "bias", (N,), f32, dev)
    prow = _maybe(row_scale, "row_scale", (M,), f32, dev)
    act_code = _act(act)
    du = _new(stream, out, dtype, dev)
    dx = _new(stream, (M, K), dtype, dev) if need_dx else None
    dw = _new(stream, (N, K), dtype, dev) if need_dw else None
    dbias = _new(stream, (N,), f32, dev) if need_dbias else None
    dcol = _new(stream, (N,), f32, dev) if need_dcol_scale else None
    if not need_dx:
        pw = w8 = None
    if not need_dw:
        px = x8 = None
    at = [p or 0 for p in (px, pw, x8 and x8.q, w8 and w8.q)]
    outputs = (GRAD_DX * need_dx + GRAD_DW * need_dw + GRAD_SUMS * (need_dbias or need_dcol_scale)
               + GRAD_DU * (du.data_ptr() % 16 == 0) + GRAD_ALIGNED * all(p % 16 == 0 for p in at))
    scales = [0 if v is None else (-(-K // v.group) or 1 if v.group else 1) for v in (x8, w8)]
    need = _size_of("dora_matmul_backward_int8_scales_workspace_size", M, N, K, code, outputs, *scales)
    workspace = _space(workspace, need, stream, dev)
    ref = [None if v is None else ctypes.byref(v) for v in (u8, x8, w8)]
    _call_on(dev, "dora_matmul_backward_int8", dy.data_ptr(), pu, ref[0], px, ref[1], pw, ref[2], code, M, N, K, prow,
             pcol, pbias, act_code, _addr(du), _addr(dx), _addr(dw), _addr(dbias), _addr(dcol), _addr(workspace), need,
             _raw_stream(stream, dev))
    return dx, dw, dbias, dcol, du
