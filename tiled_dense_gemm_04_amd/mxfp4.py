"""MXFP4 (4-bit microscaled) matrices: quantiser, inverse, products and their autograd forms.

Argument marshalling for the mxfp4_* entry points of ``include/tgemm_ops.h``, as the package's
other wrappers. An MXFP4 matrix of R x K values is a pair (codes, scale) of uint8 device
tensors: codes (R, 16 ceil(K/32)), two E2M1 codes a byte, zero past K; scale (R, ceil(K/32)),
E8M0, in rows padded to 16 bytes where this module allocates them (the fast kernels' alignment).
"""
from __future__ import annotations

import contextlib
import ctypes

from . import (SELECT_NOOP, SELECT_ZERO_FILL, TGEMM_OK, TgemmError, _as_stored, _dense_2d, _operand, lib,  # noqa: F401
               matmul)

MX_BLOCK = 32
MX_BLOCK_BYTES = 16
MX_MAX_DIM = (1 << 31) - 512         # TGEMM_MX_MAX_DIM
MX_GENERIC, MX_SKINNY, MX_128, MX_256 = range(4)   # TGEMM_MX_*
MX_SKINNY_ROWS = 64

_i64, _p, _i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
_GEMM = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _i32, _p]
_GEMM_F16 = [_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _i32, _p]
SIGNATURES = {
    "mxfp4_quant": (_i32, [_i64, _i64, _p, _i64] + [_p, _i64] * 4 + [_p]),
    "mxfp4_dequant": (_i32, [_i64, _i64] + [_p, _i64] * 3 + [_p]),
    "mxfp4_gemm": (_i32, _GEMM),
    "mxfp4_gemm_cfg": (_i32, [_i32] + _GEMM),
    "mxfp4_gemm_f16": (_i32, _GEMM_F16),
    "mxfp4_gemm_f16_cfg": (_i32, [_i32] + _GEMM_F16),
    "mxfp4_select_config": (_i32, [_i32, _i64, _i64, _i64] + [_p, _i64] * 5),
}


def _call(name, args, device, library=None):
    """The library's entry point on ``device`` (made current for the call if it is not)."""
    import torch
    fn = getattr(library or lib(), name)
    if torch.cuda.current_device() == device.index:
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def _stream(stream, device):
    import torch
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _allocating(stream, device):
    """Context in which a tensor made for a call on ``stream`` is allocated: on that stream, so
    that neither the memory's former nor its next user is on another one."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream)


def _rows_of_bytes(t, name):
    """(rows, bytes per row, row stride) of a 2-D uint8 device tensor with contiguous rows."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.uint8:
        raise TypeError(f"{name} must be uint8, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    rows, cols = t.shape
    if rows == 0 or cols == 0:
        return rows, cols, max(1, cols)
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows (stride(1) == 1)")
    return rows, cols, t.stride(0) if rows > 1 else cols


def _matrix(codes, scale, name):
    """(rows, blocks, code stride, scale stride) of an MXFP4 matrix."""
    rows, nbytes, ldq = _rows_of_bytes(codes, name)
    srows, kb, lds = _rows_of_bytes(scale, f"scale of {name}")
    if nbytes != kb * MX_BLOCK_BYTES or srows != rows:
        raise ValueError(f"{name}: codes {tuple(codes.shape)} and scale {tuple(scale.shape)} do not belong together "
                         f"(rows of {MX_BLOCK_BYTES} bytes per block of {MX_BLOCK})")
    if codes.device != scale.device:
        raise ValueError(f"{name}: codes and scale must be on the same device")
    if rows <= 1:  # one row: its stride is only its length (which the fast kernels want padded)
        lds = -(-lds // 16) * 16
    return rows, kb, max(MX_BLOCK_BYTES, ldq), max(1, lds)


def mxfp4_empty(rows: int, k: int, device):
    """Uninitialised (codes, scale) of an MXFP4 matrix of rows x k values."""
    import torch
    kb = -(-k // MX_BLOCK)
    pad = -(-kb // 16) * 16
    codes = torch.empty((rows, kb * MX_BLOCK_BYTES), dtype=torch.uint8, device=device)
    scale = torch.empty((rows, pad), dtype=torch.uint8, device=device)
    return codes, scale if pad == kb else scale[:, :kb]


def mxfp4_quant(x, dims: str = "rows", stream=None, library=None):
    """MXFP4 of fp16 x (R, K): ``dims`` "rows" gives (codes, scale) of x with blocks along K,
    "cols" those of x^T (K x R, blocks along R), "both" all four in one pass over x."""
    R, K, ldx = _operand(x, "x")
    if dims not in ("rows", "cols", "both"):
        raise ValueError(f"dims must be 'rows', 'cols' or 'both', got {dims!r}")
    out, args = (), []
    for want, rows, k in ((dims != "cols", R, K), (dims != "rows", K, R)):
        if want:
            with _allocating(stream, x.device):
                q, s = mxfp4_empty(rows, k, x.device)
            out += (q, s)
            args += [q.data_ptr(), max(MX_BLOCK_BYTES, q.shape[1]), s.data_ptr(), max(1, -(-s.shape[1] // 16) * 16)]
        else:
            args += [None, 0, None, 0]
    rc = _call("mxfp4_quant", (R, K, x.data_ptr(), ldx, *args, _stream(stream, x.device)), x.device, library)
    if rc != TGEMM_OK:
        raise TgemmError(rc, "mxfp4_quant")
    return out


def mxfp4_dequant(codes, scale, k: int, out=None, stream=None, library=None):
    """The fp16 values (R, k) of an MXFP4 matrix whose rows hold k values."""
    import torch
    R, kb, ldq, lds = _matrix(codes, scale, "codes")
    if -(-k // MX_BLOCK) != kb:
        raise ValueError(f"rows of {kb} blocks do not hold k = {k} values")
    if out is None:
        with _allocating(stream, codes.device):
            out = torch.empty((R, k), dtype=torch.float16, device=codes.device)
    Ro, Ko, ldo = _operand(out, "out")
    if (Ro, Ko) != (R, k):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(R, k)}")
    if out.device != codes.device:
        raise ValueError("codes and out must be on the same device")
    rc = _call("mxfp4_dequant", (R, k, codes.data_ptr(), ldq, scale.data_ptr(), lds, out.data_ptr(), ldo,
                                 _stream(stream, codes.device)), codes.device, library)
    if rc != TGEMM_OK:
        raise TgemmError(rc, "mxfp4_dequant")
    return out


def _output(c, M, N, device, stream):
    import torch
    if c is None:
        with _allocating(stream, device):
            return torch.empty((M, N), dtype=torch.float16, device=device), max(1, N)
    Mc, Nc, ldc = _operand(c, "c")
    if (Mc, Nc) != (M, N):
        raise ValueError(f"c has shape {tuple(c.shape)}, expected {(M, N)}")
    if c.device != device:
        raise ValueError("all operands must be on the same device")
    return c, ldc


def mxfp4_gemm(a, scale_a, b, scale_b, c=None, relu: bool = False, stream=None, cfg: int | None = None, library=None):
    """C = ReLU?(A @ B^T) of two MXFP4 matrices, A (M x K) and B (N x K); c: (M, N) fp16
    (allocated if None). ``cfg`` forces a kernel (MX_*)."""
    M, kb, lda, ldsa = _matrix(a, scale_a, "a")
    N, kb2, ldb, ldsb = _matrix(b, scale_b, "b")
    if kb != kb2:
        raise ValueError(f"inner dimensions differ: rows of {kb} and {kb2} blocks")
    if a.device != b.device:
        raise ValueError("all operands must be on the same device")
    c, ldc = _output(c, M, N, a.device, stream)
    args = (M, N, kb * MX_BLOCK, a.data_ptr(), lda, scale_a.data_ptr(), ldsa, b.data_ptr(), ldb, scale_b.data_ptr(),
            ldsb, c.data_ptr(), ldc, int(relu), _stream(stream, a.device))
    rc = (_call("mxfp4_gemm", args, a.device, library) if cfg is None
          else _call("mxfp4_gemm_cfg", (cfg, *args), a.device, library))
    if rc != TGEMM_OK:
        raise TgemmError(rc, "mxfp4_gemm" if cfg is None else f"mxfp4_gemm_cfg[{cfg}]")
    return c


def mxfp4_gemm_f16(a, b, scale_b, c=None, relu: bool = False, stream=None, cfg: int | None = None, library=None):
    """C = ReLU?(a @ W^T) of fp16 a (M, K) and an MXFP4 weight W (N x K values decoded to
    fp16); c: (M, N) fp16 (allocated if None). ``cfg`` forces a kernel (MX_*)."""
    M, K, lda = _operand(a, "a")
    N, kb, ldb, ldsb = _matrix(b, scale_b, "b")
    if -(-K // MX_BLOCK) != kb:
        raise ValueError(f"inner dimensions differ: a has {K} columns, b rows of {kb} blocks")
    if a.device != b.device:
        raise ValueError("all operands must be on the same device")
    c, ldc = _output(c, M, N, a.device, stream)
    if M == 1 and lda % 8:  # one row: its stride is only its length (which the fast kernels want padded)
        lda = -(-lda // 8) * 8
    args = (M, N, K, a.data_ptr(), lda, b.data_ptr(), ldb, scale_b.data_ptr(), ldsb, c.data_ptr(), ldc, int(relu),
            _stream(stream, a.device))
    rc = (_call("mxfp4_gemm_f16", args, a.device, library) if cfg is None
          else _call("mxfp4_gemm_f16_cfg", (cfg, *args), a.device, library))
    if rc != TGEMM_OK:
        raise TgemmError(rc, "mxfp4_gemm_f16" if cfg is None else f"mxfp4_gemm_f16_cfg[{cfg}]")
    return c


def mxfp4_select_config(M, N, K, f16_a: bool = False, A=256, lda=None, SA=256, ldsa=None, B=256, ldb=None, SB=256,
                        ldsb=None, C=256, ldc=None) -> int:
    """The kernel (MX_*) a product takes; pointers are only looked at for null and alignment."""
    kb = max(1, -(-K // MX_BLOCK))
    pad = -(-kb // 16) * 16
    lda = (max(1, K) if f16_a else kb * MX_BLOCK_BYTES) if lda is None else lda
    ldsa = pad if ldsa is None else ldsa
    ldb = kb * MX_BLOCK_BYTES if ldb is None else ldb
    ldsb = pad if ldsb is None else ldsb
    ldc = max(1, N) if ldc is None else ldc
    return int(lib().mxfp4_select_config(int(f16_a), M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc))


def mxfp4_linear(x, w_codes, scale_w, relu: bool = False, out=None, stream=None):
    """y = x W^T with W (N x K) in MXFP4: x (M x K fp16) is quantised along its rows, then
    multiplied with mxfp4_gemm, both in the library on one stream."""
    q, s = mxfp4_quant(x, "rows", stream=stream)
    return mxfp4_gemm(q, s, w_codes, scale_w, c=out, relu=relu, stream=stream)


def _row_major(x):
    """A gradient as the library takes it: rows contiguous (a copy for any other view)."""
    x = _dense_2d(x)
    return x if x.shape[1] <= 1 or x.stride(1) == 1 else x.contiguous()


def autograd_functions():
    import torch
    from torch.autograd.function import once_differentiable

    class Mxfp4LinearFunction(torch.autograd.Function):
        """y = q(x) q(w)^T for fp16 x (M, K) and w (N, K), every product of the step on MXFP4
        operands quantised along its own inner dimension: dx = q(dy) q(w^T)^T over N, dw =
        q(dy^T) q(x^T)^T over M (the quantiser's own gradient is taken as one). Each tensor is
        quantised along both axes in one pass; the backward keeps 4-bit copies only."""

        @staticmethod
        def forward(ctx, x, w):
            if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
                raise ValueError(f"x {tuple(x.shape)} and w {tuple(w.shape)} must be (M, K) and (N, K)")
            x, w = _row_major(x), _row_major(w)
            xq = mxfp4_quant(x, "both" if ctx.needs_input_grad[1] else "rows")
            wq = mxfp4_quant(w, "both" if ctx.needs_input_grad[0] else "rows")
            ctx.save_for_backward(*xq[2:], *wq[2:])
            return mxfp4_gemm(*xq[:2], *wq[:2])

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            saved = ctx.saved_tensors
            need_x, need_w = ctx.needs_input_grad
            dims = "both" if need_x and need_w else "rows" if need_x else "cols"
            q = mxfp4_quant(_row_major(dy), dims)
            dx = mxfp4_gemm(*q[:2], *saved[-2:]) if need_x else None
            dw = mxfp4_gemm(*q[-2:], *saved[:2]) if need_w else None
            return dx, dw

    class Mxfp4WeightFunction(torch.autograd.Function):
        """y = x W^T for fp16 x (M, K) and a frozen MXFP4 weight (N x K); dx = dy W with the
        weight decoded to fp16 (the codes and scales have no gradient)."""

        @staticmethod
        def forward(ctx, x, codes, scale):
            x = _row_major(x)
            ctx.save_for_backward(codes, scale)
            ctx.k = x.shape[1]
            return mxfp4_gemm_f16(x, codes, scale)

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            if not ctx.needs_input_grad[0]:
                return None, None, None
            codes, scale = ctx.saved_tensors
            return matmul(_row_major(dy), mxfp4_dequant(codes, scale, ctx.k)), None, None

    return {"Mxfp4LinearFunction": Mxfp4LinearFunction, "Mxfp4WeightFunction": Mxfp4WeightFunction}
