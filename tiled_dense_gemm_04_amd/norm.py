"""The root-mean-square norm with the residual's addition: argument marshalling for the rmsnorm_*
entry points of ``include/tgemm_ops.h``, and its autograd form.

h = x + residual, rounded to the residual's type (h = x without one), y = h w / sqrt(mean h^2 + eps).
``rmsnorm`` gives y in fp16, ``rmsnorm_fp8_block`` the E4M3 codes and scales that ``gemm_fp8_block``
takes, both beside h where there is a residual.
"""
from __future__ import annotations

import ctypes
import functools

from . import FP8_BLOCK, TGEMM_OK, TgemmError, _operand, _operand8, _scale_operand, lib
from .mxfp4 import _allocating, _call, _row_major, _stream
from .newton_schulz import DTYPE_F16, DTYPE_F32

NORM_MAX_K = 16384           # TGEMM_NORM_MAX_K

_i64, _p, _i32, _f = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "rmsnorm_f16": (_i32, [_i64, _i64, _p, _i64, _p, _i64, _i32, _p, _i32, _f, _p, _i64, _p, _i64, _p, _i64, _p, _p]),
    "rmsnorm_f16_backward_workspace_bytes": (_i64, [_i64, _i64]),
    "rmsnorm_f16_backward": (_i32, [_i64, _i64, _p, _i64, _p, _i64, _i32, _p, _i32, _f, _p, _i64, _p, _i64, _p, _i64, _p,
                                    _p, _i64, _p]),
}


@functools.lru_cache(maxsize=None)
def _types():
    import torch
    return torch.Tensor, {torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}


def _dtype(t, name):
    """The library's number of t's type (fp16 or fp32)."""
    tensor, numbers = _types()
    if not isinstance(t, tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    number = numbers.get(t.dtype)
    if number is None:
        raise TypeError(f"{name} must be float16 or float32, got {t.dtype}")
    return number


def _typed_operand(t, name, shape, device):
    """(type, row stride) of a 2-D fp16 or fp32 device tensor of `shape` with contiguous rows."""
    dtype = _dtype(t, name)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    rows, cols = shape
    if t.is_contiguous():  # (an empty one is)
        return dtype, cols or 1
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major (stride(1) == 1)")
    return dtype, t.stride(0) if rows > 1 else max(1, cols)


def _weight(w, K, device):
    dtype = _dtype(w, "weight")
    if w.shape != (K,):
        raise ValueError(f"weight has shape {tuple(w.shape)}, expected {(K,)}")
    if w.device != device:
        raise ValueError("weight must be on x's device")
    if not w.is_contiguous():
        raise ValueError("weight must be contiguous")
    return dtype


def _new(like, shape, dtype, stream):
    """An uninitialised tensor on ``like``'s device, allocated on the call's stream; like itself gives
    the shape where it is contiguous (the cheapest allocation)."""
    import torch
    if stream is None:
        if like.shape == shape and like.is_contiguous():
            return torch.empty_like(like) if like.dtype == dtype else torch.empty_like(like, dtype=dtype)
        return torch.empty(shape, dtype=dtype, device=like.device)
    with _allocating(stream, like.device):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _residual(residual, residual_out, shape, device, stream):
    """(type, row stride, the updated residual, its row stride), the latter allocated if None."""
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        return 0, 0, None, 0
    dtype, ld = _typed_operand(residual, "residual", shape, device)
    if residual_out is None:
        return dtype, ld, _new(residual, shape, residual.dtype, stream), shape[1] or 1
    out_dtype, ldo = _typed_operand(residual_out, "residual_out", shape, device)
    if out_dtype != dtype:
        raise TypeError("residual_out must have the residual's type")
    return dtype, ld, residual_out, ldo


def _norm(x, ldx, weight, residual, eps, y, ldy, q, ldq, scale, residual_out, stream, library):
    """One call on checked x and outputs; returns the updated residual (None without a residual)."""
    shape, device = x.shape, x.device
    R, K = shape
    w_dtype = _weight(weight, K, device)
    r_dtype, ldr, residual_out, ldro = _residual(residual, residual_out, shape, device, stream)
    rc = _call("rmsnorm_f16", (R, K, x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr, r_dtype,
                               weight.data_ptr(), w_dtype, eps, None if residual is None else residual_out.data_ptr(), ldro,
                               None if y is None else y.data_ptr(), ldy, None if q is None else q.data_ptr(), ldq,
                               None if q is None else scale.data_ptr(), _stream(stream, device)), device, library)
    if rc != TGEMM_OK:
        raise TgemmError(rc, "rmsnorm_f16")
    return residual_out


def rmsnorm(x, weight, residual=None, eps: float = 1e-6, out=None, residual_out=None, stream=None, library=None):
    """The norm of fp16 x (R, K) in fp16: y, or (y, h) with a ``residual`` (fp16 or fp32; h = x +
    residual in its type). ``weight``: (K,) fp16 or fp32. ``out``: y's tensor (x itself to replace it);
    ``residual_out``: h's (the residual itself to update it in place); allocated if None. K is at most
    NORM_MAX_K."""
    import torch
    R, K, ldx = _operand(x, "x")
    if out is None:
        out, ldy = _new(x, x.shape, torch.float16, stream), K or 1
    else:
        Ry, Ky, ldy = _operand(out, "out")
        if (Ry, Ky) != (R, K):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(R, K)}")
        if out.device != x.device:
            raise ValueError("x and out must be on the same device")
    h = _norm(x, ldx, weight, residual, eps, out, ldy, None, 0, None, residual_out, stream, library)
    return out if residual is None else (out, h)


def rmsnorm_fp8_block(x, weight, residual=None, eps: float = 1e-6, q=None, scale=None, residual_out=None, stream=None,
                      library=None):
    """The norm as E4M3 codes (R, K) uint8 and float32 scales (R, ceil(K/128)) per 1 x 128 block, made
    from the float32 y in the same pass: (q, scale), or (q, scale, h) with a ``residual``. Arguments as
    ``rmsnorm``; the result goes to ``gemm_fp8_block``."""
    import torch
    R, K, ldx = _operand(x, "x")
    blocks = -(-K // FP8_BLOCK)
    if q is None:
        q, ldq = _new(x, x.shape, torch.uint8, stream), K or 1
    else:
        Rq, Kq, ldq = _operand8(q, "q")
        if (Rq, Kq) != (R, K):
            raise ValueError(f"q has shape {tuple(q.shape)}, expected {(R, K)}")
    if scale is None:
        scale = _new(x, (R, blocks), torch.float32, stream)
    else:
        _scale_operand(scale, (R, blocks), "scale")
    if q.device != x.device or scale.device != x.device:
        raise ValueError("x, q and scale must be on the same device")
    h = _norm(x, ldx, weight, residual, eps, None, 0, q, ldq, scale, residual_out, stream, library)
    return (q, scale) if residual is None else (q, scale, h)


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(R, K):
    n = int(lib().rmsnorm_f16_backward_workspace_bytes(R, K))
    if n < 0:
        raise TgemmError(n, "rmsnorm_f16_backward_workspace_bytes")
    return n


def _rows(t, name, dtypes):
    """t itself where its rows are contiguous and apart, else a copy (a broadcast gradient)."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.is_contiguous():
        return t
    rows, cols = t.shape
    ld, step = t.stride()
    return t if (cols <= 1 or step == 1) and (rows <= 1 or ld >= cols) else t.contiguous()


def _ld(t):
    """Row stride of a 2-D tensor with contiguous rows, as the library takes it."""
    rows, cols = t.shape
    return cols or 1 if rows <= 1 or t.is_contiguous() else t.stride(0)


def autograd_functions():
    import torch
    f16, f32 = torch.float16, torch.float32

    class RmsNormFunction(torch.autograd.Function):
        """(x, weight, residual or None, eps) -> y, or (y, h) with a residual, for fp16 x (R, K); the
        backward pass reads h. The residual's gradient is x's in the residual's type."""

        @staticmethod
        def forward(ctx, x, weight, residual, eps):
            x = _row_major(x, "x")
            y = _new(x, x.shape, f16, None)
            weight = weight.contiguous()
            if residual is not None:
                residual = _rows(residual, "residual", (f16, f32))
            h = _norm(x, _ld(x), weight, residual, eps, y, x.shape[1] or 1, None, 0, None, None, None, None)
            kept = x if h is None else h
            ctx.save_for_backward(kept, weight)
            ctx.saved = kept.shape, kept.dtype, kept.device, weight.dtype, weight.device
            ctx.eps = eps
            ctx.set_materialize_grads(False)
            return y if h is None else (y, h)

        @staticmethod
        def backward(ctx, dy, dh=None):
            if torch.is_grad_enabled():
                raise RuntimeError("RmsNormFunction has no second derivative (create_graph=True)")
            h, weight = ctx.saved_tensors
            shape, dtype, device = h.shape, h.dtype, h.device
            # the library takes addresses
            if (shape, dtype, device, weight.dtype, weight.device) != ctx.saved or weight.shape != shape[1:]:
                raise RuntimeError("a saved-tensor hook returned another tensor than the forward pass saved")
            need_x, need_w, need_r, _ = ctx.needs_input_grad
            if dy is None:  # nothing came back through y
                if dh is None:
                    return None, None, None, None
                return dh.to(f16) if need_x else None, torch.zeros_like(weight) if need_w else None, \
                    dh if need_r else None, None
            h, weight, dy = _rows(h, "h", (dtype,)), weight.contiguous(), _rows(dy, "dy", (f16,))
            R, K = shape
            dx = _new(dy, shape, f16, None)
            dr = _new(dy, shape, f32, None) if need_r and dtype == f32 else None
            dw = workspace = None
            need = 0
            if need_w:
                dw = torch.empty_like(weight)
                need = _workspace_bytes(R, K)
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
            ld = K or 1
            if dh is not None:
                dh = _rows(dh, "dh", (dtype,))
            rc = _call("rmsnorm_f16_backward",
                       (R, K, dy.data_ptr(), _ld(dy), h.data_ptr(), _ld(h), DTYPE_F32 if dtype == f32 else DTYPE_F16,
                        weight.data_ptr(), DTYPE_F32 if weight.dtype == f32 else DTYPE_F16, ctx.eps,
                        None if dh is None else dh.data_ptr(), 0 if dh is None else _ld(dh), dx.data_ptr(), ld,
                        None if dr is None else dr.data_ptr(), ld, dw.data_ptr() if need_w else None,
                        workspace.data_ptr() if need else None, need, _stream(None, device)), device)
            if rc != TGEMM_OK:
                raise TgemmError(rc, "rmsnorm_f16_backward")
            if need_r and dr is None:
                dr = dx
            return dx if need_x else None, dw, dr if need_r else None, None

    return {"RmsNormFunction": RmsNormFunction}
