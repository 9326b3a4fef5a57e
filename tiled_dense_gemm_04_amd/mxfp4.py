"""MXFP4 (4-bit microscaled) matrices: quantiser, inverse, products and their autograd forms.

Argument marshalling for the mxfp4_* entry points of ``include/tgemm_ops.h``, as the package's
other wrappers. An MXFP4 matrix of R x K values is a pair (codes, scale) of uint8 device
tensors: codes (R, 16 ceil(K/32)), two E2M1 codes a byte, zero past K; scale (R, ceil(K/32)),
E8M0, in rows padded to 16 bytes where this module allocates them (the fast kernels' alignment).
A copy of such a scale (``clone``, ``contiguous``, a checkpoint) has its rows close together: every
operator takes it, but a product on the tile kernels lays it out again in every call: a program that
loads a weight copies it into ``mxfp4_empty``'s tensors.
"""
from __future__ import annotations

import contextlib
import ctypes

from . import TGEMM_OK, TgemmError, _operand, lib, workspace_for

MX_BLOCK = 32
MX_BLOCK_BYTES = 16
MX_MAX_DIM = (1 << 31) - 512         # TGEMM_MX_MAX_DIM
MX_GENERIC, MX_SKINNY, MX_128, MX_256, MX_64 = range(5)   # TGEMM_MX_*
MX_SKINNY_ROWS = 256
MX_ALIGNED = 256                     # stands for an aligned pointer where only the choice is asked for
MX_MAX_LDS = 1 << 23                 # the largest row stride of scales and codes in the tile kernels

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
    if torch._C._cuda_getDevice() == device.index:
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


def _matrix(codes, scale, name):
    """(rows, blocks, code stride, scale stride, device) of an MXFP4 matrix."""
    import torch
    for t, part in ((codes, name), (scale, f"scale of {name}")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{part} must be a torch.Tensor")
        if t.dtype != torch.uint8:
            raise TypeError(f"{part} must be uint8, got {t.dtype}")
        if t.dim() != 2:
            raise ValueError(f"{part} must be 2-D")
        if not t.is_cuda:
            raise ValueError(f"{part} must be a device tensor")
    (rows, nbytes), (srows, kb) = codes.shape, scale.shape
    if nbytes != kb * MX_BLOCK_BYTES or srows != rows:
        raise ValueError(f"{name}: codes {tuple(codes.shape)} and scale {tuple(scale.shape)} do not belong together "
                         f"(rows of {MX_BLOCK_BYTES} bytes per block of {MX_BLOCK})")
    device = codes.device
    if scale.device != device:
        raise ValueError(f"{name}: codes and scale must be on the same device")
    if rows == 0 or kb == 0:
        return rows, kb, max(MX_BLOCK_BYTES, nbytes), max(1, kb), device
    (ldq, cq), (lds, cs) = codes.stride(), scale.stride()
    if cq != 1 or (cs != 1 and kb > 1):
        raise ValueError(f"{name} must have contiguous rows (stride(1) == 1)")
    if rows == 1:  # one row: its stride is only its length (for the scales padded as the fast kernels want it)
        return 1, kb, nbytes, -(-kb // 16) * 16, device
    return rows, kb, ldq, lds, device


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
    device = x.device
    out, args = (), []
    for want, rows, k in ((dims != "cols", R, K), (dims != "rows", K, R)):
        if want:
            if stream is None:
                q, s = mxfp4_empty(rows, k, device)
            else:
                with _allocating(stream, device):
                    q, s = mxfp4_empty(rows, k, device)
            kb = -(-k // MX_BLOCK)
            out += (q, s)
            args += (q.data_ptr(), max(1, kb) * MX_BLOCK_BYTES, s.data_ptr(), max(1, -(-kb // 16) * 16))
        else:
            args += (None, 0, None, 0)
    rc = _call("mxfp4_quant", (R, K, x.data_ptr(), ldx, *args, _stream(stream, device)), device, library)
    if rc != TGEMM_OK:
        raise TgemmError(rc, "mxfp4_quant")
    return out


def _output(c, M, N, device, stream, name="c"):
    """The fp16 output (allocated on the call's stream if None) and its row stride."""
    if c is None:
        import torch
        if stream is None:
            return torch.empty((M, N), dtype=torch.float16, device=device), N or 1
        with _allocating(stream, device):
            return torch.empty((M, N), dtype=torch.float16, device=device), N or 1
    Mc, Nc, ldc = _operand(c, name)
    if (Mc, Nc) != (M, N):
        raise ValueError(f"{name} has shape {tuple(c.shape)}, expected {(M, N)}")
    if c.device != device:
        raise ValueError("all operands must be on the same device")
    return c, ldc


def mxfp4_dequant(codes, scale, k: int, out=None, stream=None, library=None):
    """The fp16 values (R, k) of an MXFP4 matrix whose rows hold k values."""
    R, kb, ldq, lds, device = _matrix(codes, scale, "codes")
    if -(-k // MX_BLOCK) != kb:
        raise ValueError(f"rows of {kb} blocks do not hold k = {k} values")
    out, ldo = _output(out, R, k, device, stream, "out")
    rc = _call("mxfp4_dequant", (R, k, codes.data_ptr(), ldq, scale.data_ptr(), lds, out.data_ptr(), ldo,
                                 _stream(stream, device)), device, library)
    if rc != TGEMM_OK:
        raise TgemmError(rc, "mxfp4_dequant")
    return out


def _on_tiles(library, *args) -> bool:
    """Whether a product's choice falls on a tile kernel (args: mxfp4_select_config's)."""
    return library.mxfp4_select_config(*args) in (MX_64, MX_128, MX_256)


def _worth_laying_out(M, N, kb) -> bool:
    """Whether a product whose scales are not in pieces takes longer on the generic kernel (about 7
    us, and 0.75 more per block of 32 k in each round of 128 x 128 tiles) than a copy of the scales
    and the tiles: 300 x 300 x 132 11 us against 9, 260 15 and 9.5, 516 22 and 11; 4096 x 4096 x 36
    37 and 13; the copy takes the host another 9 us."""
    return (kb + 8) * -(-(-(-M // 128) * -(-N // 128)) // 256) >= 24


def _laid_out(scale, ld, stream):
    """(scale, address, row stride) with rows in whole 16-byte pieces, as the tile kernels take them:
    itself, or a padded copy made on the call's stream."""
    import torch
    at = scale.data_ptr()
    if not (ld | at) & 15:
        return scale, at, ld
    rows, kb = scale.shape
    pad = -(-kb // 16) * 16
    with _allocating(stream, scale.device):
        out = torch.empty((rows, pad), dtype=torch.uint8, device=scale.device)
        out[:, :kb] = scale
    return out, out.data_ptr(), pad


def mxfp4_gemm(a, scale_a, b, scale_b, c=None, relu: bool = False, stream=None, cfg: int | None = None, library=None):
    """C = ReLU?(A @ B^T) of two MXFP4 matrices, A (M x K) and B (N x K); c: (M, N) fp16
    (allocated if None). ``cfg`` forces a kernel (MX_*)."""
    M, kb, lda, ldsa, device = _matrix(a, scale_a, "a")
    N, kb2, ldb, ldsb, device_b = _matrix(b, scale_b, "b")
    if kb != kb2:
        raise ValueError(f"inner dimensions differ: rows of {kb} and {kb2} blocks")
    if device_b != device:
        raise ValueError("all operands must be on the same device")
    sa, sb = scale_a.data_ptr(), scale_b.data_ptr()
    if ((sa | ldsa | sb | ldsb) & 15 and cfg is None and _worth_laying_out(M, N, kb)
            and _on_tiles(library or lib(), 0, M, N, kb * MX_BLOCK, a.data_ptr(), lda, MX_ALIGNED, MX_MAX_LDS,
                          b.data_ptr(), ldb, MX_ALIGNED, MX_MAX_LDS, MX_ALIGNED, N)):
        scale_a, sa, ldsa = _laid_out(scale_a, ldsa, stream)
        scale_b, sb, ldsb = _laid_out(scale_b, ldsb, stream)
    c, ldc = _output(c, M, N, device, stream)
    args = (M, N, kb * MX_BLOCK, a.data_ptr(), lda, sa, ldsa, b.data_ptr(), ldb, sb, ldsb, c.data_ptr(), ldc, int(relu),
            _stream(stream, device))
    rc = (_call("mxfp4_gemm", args, device, library) if cfg is None
          else _call("mxfp4_gemm_cfg", (cfg, *args), device, library))
    if rc != TGEMM_OK:
        raise TgemmError(rc, "mxfp4_gemm" if cfg is None else f"mxfp4_gemm_cfg[{cfg}]")
    return c


def _padded_rows(x):
    """x (M, K) with zeros to a multiple of 8 columns, in rows of that length."""
    import torch
    M, K = x.shape
    y = torch.empty((M, -(-K // 8) * 8), dtype=x.dtype, device=x.device)
    y[:, :K] = x
    if K % 8:
        y[:, K:] = 0
    return y


def mxfp4_gemm_f16(a, b, scale_b, c=None, relu: bool = False, stream=None, cfg: int | None = None, library=None):
    """C = ReLU?(a @ W^T) of fp16 a (M, K) and an MXFP4 weight W (N x K values decoded to
    fp16); c: (M, N) fp16 (allocated if None). ``cfg`` forces a kernel (MX_*). Where the choice
    falls on tiles that cannot take ``a`` (K or the row stride no multiple of 8, a base off 16
    bytes), its rows are copied once to ones they can (100 x 8192 x 4095: 47 us against 110 on the
    generic kernel); and the scales likewise."""
    M, K, lda = _operand(a, "a")
    N, kb, ldb, ldsb, device = _matrix(b, scale_b, "b")
    if -(-K // MX_BLOCK) != kb:
        raise ValueError(f"inner dimensions differ: a has {K} columns, b rows of {kb} blocks")
    if a.device != device:
        raise ValueError("all operands must be on the same device")
    at, sb = a.data_ptr(), scale_b.data_ptr()
    odd, close = (K | lda) & 7 or at & 15, (sb | ldsb) & 15
    if (odd or close) and cfg is None and (not close or _worth_laying_out(M, N, kb)):
        k8 = -(-K // 8) * 8
        if _on_tiles(library or lib(), 1, M, N, k8, MX_ALIGNED, k8, None, 0, b.data_ptr(), ldb, MX_ALIGNED, MX_MAX_LDS,
                     MX_ALIGNED, N):
            if odd:
                with _allocating(stream, device):
                    a = _padded_rows(a)
                M, K, lda = _operand(a, "a")
                at = a.data_ptr()
            scale_b, sb, ldsb = _laid_out(scale_b, ldsb, stream)
    c, ldc = _output(c, M, N, device, stream)
    if M == 1 and lda % 8:  # one row: its stride is only its length (which the fast kernels want padded)
        lda = -(-lda // 8) * 8
    args = (M, N, K, at, lda, b.data_ptr(), ldb, sb, ldsb, c.data_ptr(), ldc, int(relu), _stream(stream, device))
    rc = (_call("mxfp4_gemm_f16", args, device, library) if cfg is None
          else _call("mxfp4_gemm_f16_cfg", (cfg, *args), device, library))
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


def _row_major(x, name):
    """A 2-D fp16 device tensor as the library takes it: rows contiguous (a copy for any other
    view)."""
    import torch
    if not isinstance(x, torch.Tensor) or x.dtype != torch.float16 or x.dim() != 2 or not x.is_cuda:
        raise TypeError(f"{name} must be a 2-D float16 device tensor")
    rows, cols = x.shape
    ld, step = x.stride()
    return x if (cols <= 1 or step == 1) and (rows <= 1 or ld >= cols) else x.contiguous()


def _once():
    """A backward pass runs with gradients recorded only when its own gradient is wanted."""
    import torch
    if torch.is_grad_enabled():
        raise RuntimeError("the MXFP4 functions have no second derivative (create_graph=True)")


def _times_weight(dy, codes, scale, k):
    """dy @ W (M x N by N x k) with W decoded to fp16, through gemm_f16_ws as ``matmul`` runs it.
    Sizes that are no multiples of 8 are padded to ones, which the fast GEMM kernels take: W's rows
    to whole blocks (zero codes) and N with zeros; the result is the part of a wider buffer."""
    import torch
    (M, N), device = dy.shape, dy.device
    width, n8 = codes.shape[1] * 2, -(-N // 8) * 8
    if n8 != N or dy.data_ptr() % 16 or (M > 1 and dy.stride(0) % 8):
        dy = _padded_rows(dy)
    w = torch.empty((n8, width), dtype=torch.float16, device=device)
    mxfp4_dequant(codes, scale, width, out=w[:N])
    if n8 != N:
        w[N:] = 0
    dx = torch.empty((M, width), dtype=torch.float16, device=device)
    L, stream = lib(), _stream(None, device)
    need = L.tgemm_workspace_bytes(0, 0, M, width, n8)
    ws = None
    if need:  # a captured graph gets a (zeroed) workspace of its own: its replays may overlap other calls
        ws = (torch.zeros(need, dtype=torch.uint8, device=device) if torch.cuda.is_current_stream_capturing()
              else workspace_for(need, device, stream))
    rc = _call("gemm_f16_ws", (0, 0, M, width, n8, dy.data_ptr(), dy.stride(0) if M > 1 else n8 or 1, w.data_ptr(),
                               width or 1, dx.data_ptr(), width or 1, 0, ws.data_ptr() if need else None,
                               ws.numel() if need else 0, stream), device)
    if rc != TGEMM_OK:
        raise TgemmError(rc, "gemm_f16_ws")
    return dx if width == k else dx[:, :k]


class _Packed:
    """MXFP4 matrices in one allocation (a step of a linear layer makes six of them): ``add``
    plans one and returns (rows, k, code offset, code stride, scale offset, scale stride)."""

    def __init__(self, device):
        self.device, self.nbytes, self.base = device, 0, 0

    def add(self, rows, k):
        kb = -(-k // MX_BLOCK) or 1
        ldq, lds = kb * MX_BLOCK_BYTES, -(-kb // 16) * 16
        at = self.nbytes
        self.nbytes = at + rows * (ldq + lds)
        return rows, k, at, ldq, at + rows * ldq, lds

    def allocate(self):
        import torch
        self.tensor = torch.empty(self.nbytes, dtype=torch.uint8, device=self.device)
        self.base = self.tensor.data_ptr()
        return self.tensor


def _packed_quant(x, rows, cols, rows_base, cols_base):
    """Quantise x into planned matrices (None: not wanted)."""
    R, K = x.shape
    ldx = x.stride(0) if R > 1 else max(1, K)
    a = (rows_base + rows[2], rows[3], rows_base + rows[4], rows[5]) if rows else (None, 0, None, 0)
    b = (cols_base + cols[2], cols[3], cols_base + cols[4], cols[5]) if cols else (None, 0, None, 0)
    device = x.device
    rc = _call("mxfp4_quant", (R, K, x.data_ptr(), ldx, *a, *b, _stream(None, device)), device)
    if rc != TGEMM_OK:
        raise TgemmError(rc, "mxfp4_quant")


def _packed_gemm(a, a_base, b, b_base, device):
    import torch
    M, N = a[0], b[0]
    c = torch.empty((M, N), dtype=torch.float16, device=device)
    rc = _call("mxfp4_gemm", (M, N, a[1], a_base + a[2], a[3], a_base + a[4], a[5], b_base + b[2], b[3], b_base + b[4],
                              b[5], c.data_ptr(), N or 1, 0, _stream(None, device)), device)
    if rc != TGEMM_OK:
        raise TgemmError(rc, "mxfp4_gemm")
    return c


def autograd_functions():
    import torch

    class Mxfp4LinearFunction(torch.autograd.Function):
        """y = q(x) q(w)^T for fp16 x (M, K) and w (N, K), every product of the step on MXFP4
        operands quantised along its own inner dimension: dx = q(dy) q(w^T)^T over N, dw =
        q(dy^T) q(x^T)^T over M (the quantiser's own gradient is taken as one). Each tensor is
        quantised along both axes in one pass; the backward keeps 4-bit copies only."""

        @staticmethod
        def forward(ctx, x, w):
            x, w = _row_major(x, "x"), _row_major(w, "w")
            if x.shape[1] != w.shape[1] or x.device != w.device:
                raise ValueError(f"x {tuple(x.shape)} and w {tuple(w.shape)} must be (M, K) and (N, K) on one device")
            need_x, need_w = ctx.needs_input_grad
            rows, cols = _Packed(x.device), _Packed(x.device)
            xq, wq = rows.add(*x.shape), rows.add(*w.shape)
            ctx.xt = cols.add(x.shape[1], x.shape[0]) if need_w else None
            ctx.wt = cols.add(w.shape[1], w.shape[0]) if need_x else None
            kept = cols.allocate()
            rows.allocate()
            ctx.save_for_backward(kept)
            ctx.kept = kept.shape
            _packed_quant(x, xq, ctx.xt, rows.base, cols.base)
            _packed_quant(w, wq, ctx.wt, rows.base, cols.base)
            return _packed_gemm(xq, rows.base, wq, rows.base, x.device)

        @staticmethod
        def backward(ctx, dy):
            _once()
            need_x, need_w = ctx.needs_input_grad
            dy = _row_major(dy, "dy")
            tmp = _Packed(dy.device)
            M, N = dy.shape
            q = tmp.add(M, N) if need_x else None
            qt = tmp.add(N, M) if need_w else None
            tmp.allocate()
            # (the tensor itself, until both products are launched: under saved-tensor hooks, as
            # checkpointing sets them, it is a copy that nothing else owns)
            kept, = ctx.saved_tensors
            if (kept.shape, kept.dtype, kept.device, kept.is_contiguous()) != (ctx.kept, torch.uint8, dy.device, True):
                raise RuntimeError("a saved-tensor hook returned another tensor than the forward pass saved")
            _packed_quant(dy, q, qt, tmp.base, tmp.base)
            dx = _packed_gemm(q, tmp.base, ctx.wt, kept.data_ptr(), dy.device) if need_x else None
            dw = _packed_gemm(qt, tmp.base, ctx.xt, kept.data_ptr(), dy.device) if need_w else None
            return dx, dw

    class Mxfp4WeightFunction(torch.autograd.Function):
        """y = x W^T for fp16 x (M, K) and a frozen MXFP4 weight (N x K); dx = dy W with the
        weight decoded to fp16 (the codes and scales have no gradient)."""

        @staticmethod
        def forward(ctx, x, codes, scale):
            x = _row_major(x, "x")
            ctx.save_for_backward(codes, scale)
            ctx.k = x.shape[1]
            return mxfp4_gemm_f16(x, codes, scale)

        @staticmethod
        def backward(ctx, dy):
            _once()
            codes, scale = ctx.saved_tensors
            return _times_weight(_row_major(dy, "dy"), codes, scale, ctx.k), None, None

    return {"Mxfp4LinearFunction": Mxfp4LinearFunction, "Mxfp4WeightFunction": Mxfp4WeightFunction}
