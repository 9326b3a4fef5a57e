"""Newton-Schulz orthogonalisation of weight updates: the orthogonalize_* entry points of
``include/tgemm_ops.h``."""
from __future__ import annotations

import ctypes

from . import TGEMM_OK, TgemmError, lib
from .mxfp4 import _allocating, _call, _stream

DTYPE_F16, DTYPE_F32 = 0, 1          # TGEMM_DTYPE_*
NS_COEFFICIENTS = (3.4445, -4.7750, 2.0315)

_i64, _p, _i32, _f = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "orthogonalize_workspace_bytes": (_i64, [_i64, _i64, _i64]),
    "orthogonalize_f16": (_i32, [_i64, _i64, _i64, _i32, _p, _i64, _i64, _p, _i64, _i64, _i32, _f, _f, _f, _f, _p,
                                 _i64, _p]),
}


def orthogonalize_workspace_bytes(batch: int, rows: int, cols: int) -> int:
    n = int(lib().orthogonalize_workspace_bytes(batch, rows, cols))
    if n < 0:
        raise TgemmError(n, "orthogonalize_workspace_bytes")
    return n


def _stack(t, name, dtypes):
    """(batch, rows, cols, row stride, matrix stride) of a 2-D or 3-D device tensor with
    contiguous rows."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be 2-D or a 3-D stack of matrices")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    rows, cols = t.shape[-2:]
    batch = t.shape[0] if t.dim() == 3 else 1
    if t.numel() == 0:
        return batch, rows, cols, max(1, cols), rows * max(1, cols)
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be row-major (stride(-1) == 1)")
    ld = t.stride(-2) if rows > 1 else max(1, cols)
    return batch, rows, cols, ld, (t.stride(0) if batch > 1 else rows * ld)


def orthogonalize(g, steps: int = 5, scale: float = 1.0, out=None, coefficients=NS_COEFFICIENTS, workspace=None,
                  stream=None, library=None):
    """scale * NS(g) as fp16 for fp16 or fp32 g: one matrix (R, C) or a stack (batch, R, C), each
    divided by its Frobenius norm and run through ``steps`` Newton-Schulz products with
    ``coefficients``, to what float32 products give rounded once. ``out``: fp16, g's shape (allocated if None; g itself if it is fp16).
    ``workspace``: a uint8 device tensor of orthogonalize_workspace_bytes(batch, R, C), 256-byte
    aligned (allocated for the call if None)."""
    import torch
    batch, R, C, ldg, sg = _stack(g, "g", (torch.float16, torch.float32))
    if out is None:
        with _allocating(stream, g.device):
            out = torch.empty(g.shape, dtype=torch.float16, device=g.device)
    elif tuple(out.shape) != tuple(g.shape):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(g.shape)}")
    _, _, _, ldx, sx = _stack(out, "out", (torch.float16,))
    if out.device != g.device:
        raise ValueError("g and out must be on the same device")
    need = orthogonalize_workspace_bytes(batch, R, C)
    if workspace is None:
        with _allocating(stream, g.device):
            workspace = torch.empty(need, dtype=torch.uint8, device=g.device)
    elif workspace.device != g.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on g's device")
    a, b, c = coefficients
    rc = _call("orthogonalize_f16",
               (batch, R, C, DTYPE_F32 if g.dtype == torch.float32 else DTYPE_F16, g.data_ptr(), ldg, sg,
                out.data_ptr(), ldx, sx, int(steps), a, b, c, scale, workspace.data_ptr(),
                workspace.numel() * workspace.element_size(), _stream(stream, g.device)), g.device, library)
    if rc != TGEMM_OK:
        raise TgemmError(rc, "orthogonalize_f16")
    return out
