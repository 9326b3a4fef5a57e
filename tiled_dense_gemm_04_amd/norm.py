"""The root-mean-square norm with the residual's addition: argument marshalling for the rmsnorm_*
entry points of ``include/tgemm_ops.h``, and its autograd form.

h = x + residual, rounded to the residual's type (h = x without one), y = h w / sqrt(mean h^2 + eps).
``rmsnorm`` gives y in fp16, ``rmsnorm_fp8_block`` the E4M3 codes and scales that ``gemm_fp8_block``
takes, both beside h where there is a residual.
"""
from __future__ import annotations

import ctypes

from . import FP8_BLOCK, TGEMM_OK, TgemmError, _operand, _operand8, _scale_operand, lib
from .mxfp4 import _allocating, _call, _row_major, _stream
from .newton_schulz import DTYPE_F16, DTYPE_F32

NORM_MAX_K = 16384           # TGEMM_NORM_MAX_K

_i64, _p, _i32, _f = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "rmsnorm_f16": (_i32, [_i64, _i64, _p, _i64, _p, _i64, _i32, _p, _i32, _f, _p, _i64, _p, _i64, _p, _i64, _p, _p, _p]),
    "rmsnorm_f16_backward_workspace_bytes": (_i64, [_i64, _i64]),
    "rmsnorm_f16_backward": (_i32, [_i64, _i64, _p, _i64, _p, _i64, _i32, _p, _i32, _p, _p, _i64, _p, _i64, _p, _i64, _p,
                                    _p, _i64, _p]),
}


def _dtype(t, name):
    """The library's number of t's type (fp16 or fp32)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype == torch.float16:
        return DTYPE_F16
    if t.dtype == torch.float32:
        return DTYPE_F32
    raise TypeError(f"{name} must be float16 or float32, got {t.dtype}")


def _typed_operand(t, name, shape, device):
    """(type, row stride) of a 2-D fp16 or fp32 device tensor of `shape` with contiguous rows."""
    dtype = _dtype(t, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    rows, cols = shape
    if t.numel() == 0:
        return dtype, max(1, cols)
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major (stride(1) == 1)")
    return dtype, t.stride(0) if rows > 1 else max(1, cols)


def _weight(w, K, device):
    dtype = _dtype(w, "weight")
    if tuple(w.shape) != (K,):
        raise ValueError(f"weight has shape {tuple(w.shape)}, expected {(K,)}")
    if w.device != device:
        raise ValueError("weight must be on x's device")
    if K > 1 and w.stride(0) != 1:
        raise ValueError("weight must be contiguous")
    return dtype


def _norm(x, weight, residual, eps, y, q, scale, rstd, residual_out, stream, library):
    """One call; returns the updated residual (allocated if None, None without a residual)."""
    import torch
    R, K, ldx = _operand(x, "x")
    device = x.device
    w_dtype = _weight(weight, K, device)
    r_dtype = ldr = ldro = 0
    if residual is not None:
        r_dtype, ldr = _typed_operand(residual, "residual", (R, K), device)
        if residual_out is None:
            with _allocating(stream, device):
                residual_out = torch.empty((R, K), dtype=residual.dtype, device=device)
        o_dtype, ldro = _typed_operand(residual_out, "residual_out", (R, K), device)
        if o_dtype != r_dtype:
            raise TypeError("residual_out must have the residual's type")
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    ldy = ldq = 0
    if y is not None:
        Ry, Ky, ldy = _operand(y, "out")
        if (Ry, Ky) != (R, K):
            raise ValueError(f"out has shape {tuple(y.shape)}, expected {(R, K)}")
        if y.device != device:
            raise ValueError("x and out must be on the same device")
    if q is not None:
        Rq, Kq, ldq = _operand8(q, "q")
        if (Rq, Kq) != (R, K):
            raise ValueError(f"q has shape {tuple(q.shape)}, expected {(R, K)}")
        _scale_operand(scale, (R, -(-K // FP8_BLOCK)), "scale")
        if q.device != device or scale.device != device:
            raise ValueError("x, q and scale must be on the same device")

    def at(t):
        return None if t is None else t.data_ptr()

    rc = _call("rmsnorm_f16", (R, K, x.data_ptr(), ldx, at(residual), ldr, r_dtype, weight.data_ptr(), w_dtype, eps,
                               at(residual_out), ldro, at(y), ldy, at(q), ldq, at(scale), at(rstd),
                               _stream(stream, device)), device, library)
    if rc != TGEMM_OK:
        raise TgemmError(rc, "rmsnorm_f16")
    return residual_out


def rmsnorm(x, weight, residual=None, eps: float = 1e-6, out=None, residual_out=None, stream=None, library=None):
    """The norm of fp16 x (R, K) in fp16: y, or (y, h) with a ``residual`` (fp16 or fp32; h = x +
    residual in its type). ``weight``: (K,) fp16 or fp32. ``out``: y's tensor (x itself to replace it);
    ``residual_out``: h's (the residual itself to update it in place); allocated if None. K is at most
    NORM_MAX_K."""
    import torch
    if out is None:
        R, K, _ = _operand(x, "x")
        with _allocating(stream, x.device):
            out = torch.empty((R, K), dtype=torch.float16, device=x.device)
    h = _norm(x, weight, residual, eps, out, None, None, None, residual_out, stream, library)
    return out if residual is None else (out, h)


def rmsnorm_fp8_block(x, weight, residual=None, eps: float = 1e-6, q=None, scale=None, residual_out=None, stream=None,
                      library=None):
    """The norm as E4M3 codes (R, K) uint8 and float32 scales (R, ceil(K/128)) per 1 x 128 block, made
    from the float32 y in the same pass: (q, scale), or (q, scale, h) with a ``residual``. Arguments as
    ``rmsnorm``; the result goes to ``gemm_fp8_block``."""
    import torch
    R, K, _ = _operand(x, "x")
    with _allocating(stream, x.device):
        if q is None:
            q = torch.empty((R, K), dtype=torch.uint8, device=x.device)
        if scale is None:
            scale = torch.empty((R, -(-K // FP8_BLOCK)), dtype=torch.float32, device=x.device)
    h = _norm(x, weight, residual, eps, None, q, scale, None, residual_out, stream, library)
    return (q, scale) if residual is None else (q, scale, h)


def _rows(t, name, dtypes):
    """t itself where its rows are contiguous and apart, else a copy (a broadcast gradient)."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    rows, cols = t.shape
    return t if (cols <= 1 or t.stride(1) == 1) and (rows <= 1 or t.stride(0) >= cols) else t.contiguous()


def autograd_functions():
    import torch

    class RmsNormFunction(torch.autograd.Function):
        """(x, weight, residual or None, eps) -> y, or (y, h) with a residual, for fp16 x (R, K); the
        backward pass reads h and a float32 number per row. The residual's gradient is x's in the
        residual's type."""

        @staticmethod
        def forward(ctx, x, weight, residual, eps):
            x = _row_major(x, "x")
            R, K = x.shape
            y = torch.empty((R, K), dtype=torch.float16, device=x.device)
            rstd = torch.empty(R, dtype=torch.float32, device=x.device)
            weight = weight.contiguous()
            if residual is not None:
                residual = _rows(residual, "residual", (torch.float16, torch.float32))
            h = _norm(x, weight, residual, eps, y, None, None, rstd, None, None, None)
            ctx.save_for_backward(x if h is None else h, weight, rstd)
            ctx.saved = tuple((t.shape, t.dtype) for t in (x if h is None else h, weight, rstd))
            ctx.has_residual = h is not None
            ctx.set_materialize_grads(False)
            return y if h is None else (y, h)

        @staticmethod
        def backward(ctx, dy, dh=None):
            if torch.is_grad_enabled():
                raise RuntimeError("RmsNormFunction has no second derivative (create_graph=True)")
            h, weight, rstd = ctx.saved_tensors
            for t, (shape, dtype) in zip((h, weight, rstd), ctx.saved):
                if t.shape != shape or t.dtype != dtype or not t.is_cuda or t.device != h.device:
                    raise RuntimeError("a saved-tensor hook returned another tensor than the forward pass saved")
            device = h.device
            h, weight, rstd = _rows(h, "h", (h.dtype,)), weight.contiguous(), rstd.contiguous()
            R, K = h.shape
            need_x, need_w, need_r, _ = ctx.needs_input_grad
            if dy is None:  # nothing came back through y
                if dh is None:
                    return None, None, None, None
                return dh.to(torch.float16) if need_x else None, torch.zeros_like(weight) if need_w else None, \
                    dh if need_r else None, None
            dy = _rows(dy, "dy", (torch.float16,))
            dh = None if dh is None else _rows(dh, "dh", (h.dtype,))
            dx = torch.empty((R, K), dtype=torch.float16, device=device)
            dr = torch.empty_like(dx, dtype=h.dtype) if need_r and h.dtype != torch.float16 else None
            dw = torch.empty_like(weight) if need_w else None
            need = int(lib().rmsnorm_f16_backward_workspace_bytes(R, K)) if need_w else 0
            workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None

            def at(t):
                return None if t is None else t.data_ptr()

            def ld(t):
                return 0 if t is None else max(1, K) if R <= 1 else t.stride(0)

            h_dtype = DTYPE_F32 if h.dtype == torch.float32 else DTYPE_F16
            w_dtype = DTYPE_F32 if weight.dtype == torch.float32 else DTYPE_F16
            rc = _call("rmsnorm_f16_backward",
                       (R, K, dy.data_ptr(), ld(dy), h.data_ptr(), ld(h), h_dtype, weight.data_ptr(), w_dtype,
                        rstd.data_ptr(), at(dh), ld(dh), dx.data_ptr(), ld(dx), at(dr), ld(dr), at(dw), at(workspace),
                        need, _stream(None, device)), device)
            if rc != TGEMM_OK:
                raise TgemmError(rc, "rmsnorm_f16_backward")
            if need_r and dr is None:
                dr = dx
            return dx if need_x else None, dw, dr if need_r else None, None

    return {"RmsNormFunction": RmsNormFunction}
