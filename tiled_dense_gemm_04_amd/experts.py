"""An expert layer's rows: tokens sorted by expert and back, and the experts' products over the sorted
rows. Argument marshalling for the expert_* entry points of ``include/tgemm_ops.h``, and their autograd
forms. Everything that depends on the ids stays on the device: nothing here waits for the GPU, and a
whole layer can be captured into a graph.

    plan = expert_sort(ids, E)                       # ids (T, k): each token's experts
    xs = expert_gather(x, plan)                      # (T k, H): the rows of each expert together
    hs = expert_gemm_f16(xs, up, plan.offsets, relu=True)
    ys = expert_gemm_f16(hs, down, plan.offsets)
    y = expert_combine(ys, plan, weights)            # (T, H)

Sums are float32, and every result is rounded to binary16 once, as what passes between operators takes two
bytes a value: the layer above rounds its inner rows, the second product's rows and its output (with a norm
before it 4.2e-4 of its values' size from the exact one in all, where one rounding is 2.1e-4).
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import TGEMM_OK, TgemmError, _operand, lib
from .mxfp4 import _allocating, _call, _output, _row_major, _stream
from .newton_schulz import DTYPE_F16, DTYPE_F32, _stack

MAX_EXPERTS = 1024                    # TGEMM_MAX_EXPERTS
MAX_SLOTS = (1 << 26) - 1024          # TGEMM_MAX_SLOTS
INDEX_I32, INDEX_I64 = 0, 1           # TGEMM_INDEX_*
EXPERT_GENERIC, EXPERT_32, EXPERT_128, EXPERT_256, EXPERT_TILES, EXPERT_64 = range(6)   # TGEMM_EXPERT_*

_i64, _p, _i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
_GEMM = [_i32, _i64, _i64, _i64, _i64, _p, _i64, _p, _p, _i64, _i64, _p, _i64, _i32, _i32, _p]
_GEMM_TN = [_i64, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _i64, _i64, _p]
SIGNATURES = {
    "expert_sort_workspace_bytes": (_i64, [_i64, _i64, _i64]),
    "expert_sort": (_i32, [_i64, _i64, _i64, _p, _i64, _i32, _p, _p, _p, _p, _i64, _p]),
    "expert_gather_f16": (_i32, [_i64, _i64, _i64, _i64, _p, _i64, _p, _p, _i64, _p, _i64, _p]),
    "expert_combine_f16": (_i32, [_i64, _i64, _i64, _i64, _p, _i64, _p, _p, _i32, _p, _i64, _p]),
    "expert_combine_f16_backward": (_i32, [_i64, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _i32, _p, _i64, _p, _p,
                                           _i64, _p]),
    "expert_gemm_f16": (_i32, _GEMM),
    "expert_gemm_f16_cfg": (_i32, [_i32] + _GEMM),
    "expert_gemm_f16_tn": (_i32, _GEMM_TN),
    "expert_gemm_f16_tn_cfg": (_i32, [_i32] + _GEMM_TN),
    "expert_gemm_select_config": (_i32, [_i32, _i64, _i64, _i64, _i64, _i64, _p, _i64, _p, _i64, _i64]),
}


class ExpertOrder(NamedTuple):
    """Where the slots of (T, k) ids go: ``offsets`` (experts + 1), ``order`` (T k: the slot of each
    sorted row, -1 behind the last) and ``place`` (T, k: each slot's row, -1 for none), int32. The autograd
    functions take it as ``expert_sort`` wrote it, where each of the offsets[-1] rows in use has its slot: rows
    that lost theirs to a change of ``place`` are not written, and a gradient is summed over them. To leave
    slots out, give them an id of no expert before sorting."""
    offsets: "torch.Tensor"  # noqa: F821
    order: "torch.Tensor"    # noqa: F821
    place: "torch.Tensor"    # noqa: F821


def _int32(t, name, dim, device=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    if t.dim() != dim or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dim}-D device tensor")
    if device is not None and t.device != device:
        raise ValueError("all operands must be on the same device")
    return t


def _offsets(t, device, experts=None):
    """The number of experts that offsets are for."""
    _int32(t, "offsets", 1, device)
    if not 2 <= t.numel() <= MAX_EXPERTS + 1 or (experts is not None and t.numel() != experts + 1):
        raise ValueError(f"offsets has {t.numel()} elements, expected {'2 to %d' % (MAX_EXPERTS + 1) if experts is None else experts + 1}")
    return t.numel() - 1


def expert_sort(ids, experts: int, stream=None, library=None) -> ExpertOrder:
    """Sorts the slots of ids (T, k; int32 or int64, contiguous rows) by expert, stably. An id outside
    [0, experts) is a slot of no expert. experts is at most MAX_EXPERTS, T * k at most MAX_SLOTS."""
    import torch
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    if ids.dim() != 2:
        raise ValueError("ids must be 2-D (tokens, choices)")
    if not ids.is_cuda:
        raise ValueError("ids must be a device tensor")
    T, k = ids.shape
    if ids.numel() and k > 1 and ids.stride(1) != 1:
        raise ValueError("ids must be row-major (stride(1) == 1)")
    ldi = ids.stride(0) if T > 1 and ids.numel() else max(1, k)
    device = ids.device
    need = (library or lib()).expert_sort_workspace_bytes(T, k, experts)
    if need < 0:
        raise TgemmError(need, "expert_sort_workspace_bytes")
    with _allocating(stream, device):
        offsets = torch.empty(experts + 1, dtype=torch.int32, device=device)
        order = torch.empty(T * k, dtype=torch.int32, device=device)
        place = torch.empty((T, k), dtype=torch.int32, device=device)
        workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    rc = _call("expert_sort", (T, k, experts, ids.data_ptr(), ldi, INDEX_I64 if ids.dtype == torch.int64 else INDEX_I32,
                               offsets.data_ptr(), order.data_ptr(), place.data_ptr(),
                               workspace.data_ptr() if need else None, need, _stream(stream, device)), device, library)
    if rc != TGEMM_OK:
        raise TgemmError(rc, "expert_sort")
    return ExpertOrder(offsets, order, place)


def expert_gather(x, plan: ExpertOrder, out=None, zero_rest: bool = False, stream=None, library=None):
    """The rows of fp16 x (T, H) in the plan's order: (T k, H), token t's at each of its places. Rows
    behind the last one in use are left as they were (in ``out``, or uninitialised where it is
    allocated here); with ``zero_rest`` they are set to zero."""
    T, H, ldx = _operand(x, "x")
    device = x.device
    place = _int32(plan.place, "plan.place", 2, device)
    if place.shape[0] != T:
        raise ValueError(f"x has {T} rows, the plan {place.shape[0]} tokens")
    k = place.shape[1]
    out, ldo = _output(out, T * k, H, device, stream, "out")
    experts = _offsets(plan.offsets, device) if zero_rest else 0
    rc = _call("expert_gather_f16", (T, k, T * k, H, x.data_ptr(), ldx, place.data_ptr(), out.data_ptr(), ldo,
                                     plan.offsets.data_ptr() if zero_rest else None, experts, _stream(stream, device)),
               device, library)
    if rc != TGEMM_OK:
        raise TgemmError(rc, "expert_gather_f16")
    return out


def _weights(w, shape, device):
    """(address, type) of the slots' weights, fp32 or fp16 (T, k) contiguous, or None."""
    import torch
    if w is None:
        return None, DTYPE_F32
    if not isinstance(w, torch.Tensor) or w.dtype not in (torch.float32, torch.float16):
        raise TypeError("weights must be a float32 or float16 tensor")
    if tuple(w.shape) != tuple(shape):
        raise ValueError(f"weights has shape {tuple(w.shape)}, expected {tuple(shape)}")
    if w.device != device or not w.is_contiguous():
        raise ValueError("weights must be a contiguous tensor on the rows' device")
    return w.data_ptr(), DTYPE_F32 if w.dtype == torch.float32 else DTYPE_F16


def expert_combine(y, plan: ExpertOrder, weights=None, out=None, stream=None, library=None):
    """out[t] = sum_j weights[t, j] y[place[t, j]] for fp16 y (rows, H), (T, H) fp16: float32 sums in the
    order of j, rounded once. ``weights``: (T, k) fp32 or fp16 (None: ones). Slots of no expert add
    nothing."""
    rows, H, ldy = _operand(y, "y")
    device = y.device
    place = _int32(plan.place, "plan.place", 2, device)
    T, k = place.shape
    w, w_dtype = _weights(weights, (T, k), device)
    out, ldo = _output(out, T, H, device, stream, "out")
    rc = _call("expert_combine_f16", (T, k, rows, H, y.data_ptr(), ldy, place.data_ptr(), w, w_dtype, out.data_ptr(), ldo,
                                      _stream(stream, device)), device, library)
    if rc != TGEMM_OK:
        raise TgemmError(rc, "expert_combine_f16")
    return out


def _stacked(b, name):
    import torch
    if isinstance(b, torch.Tensor) and b.dim() != 3:
        raise ValueError(f"{name} must be a 3-D stack, one matrix an expert")
    return _stack(b, name, (torch.float16,))


def expert_gemm_f16(a, b, offsets, c=None, relu: bool = False, trans_b: bool = True, zero_rest: bool = False, stream=None,
                    cfg: int | None = None, library=None):
    """c[p] = ReLU?(a[p] @ op(b[e])) for the rows offsets[e] <= p < offsets[e + 1] of fp16 a (rows, K);
    b: (E, N, K) fp16, one linear layer's weight an expert, or (E, K, N) with trans_b=False; c: (rows, N)
    fp16 (allocated if None). Rows of no expert are left as they were, or from offsets[E] on set to
    zero with ``zero_rest``. ``cfg`` forces a kernel (EXPERT_*)."""
    rows, K, lda = _operand(a, "a")
    E, rb, cb, ldb, sb = _stacked(b, "b")
    N, K2 = (rb, cb) if trans_b else (cb, rb)
    if K2 != K:
        raise ValueError(f"inner dimensions differ: a is {rows}x{K}, op(b) is {K2}x{N}")
    device = a.device
    if b.device != device:
        raise ValueError("all operands must be on the same device")
    _offsets(offsets, device, E)
    c, ldc = _output(c, rows, N, device, stream)
    args = (int(trans_b), rows, E, N, K, a.data_ptr(), lda, offsets.data_ptr(), b.data_ptr(), ldb, sb, c.data_ptr(), ldc,
            int(relu), int(zero_rest), _stream(stream, device))
    rc = (_call("expert_gemm_f16", args, device, library) if cfg is None
          else _call("expert_gemm_f16_cfg", (cfg, *args), device, library))
    if rc != TGEMM_OK:
        raise TgemmError(rc, "expert_gemm_f16" if cfg is None else f"expert_gemm_f16_cfg[{cfg}]")
    return c


def expert_gemm_f16_tn(a, b, offsets, c=None, stream=None, cfg: int | None = None, library=None):
    """c[e] = a_e^T @ b_e over the expert's rows of fp16 a (rows, M) and b (rows, N): (E, M, N) fp16
    (allocated if None), zeros for an expert of no rows. ``cfg`` forces a kernel (EXPERT_*)."""
    import torch
    rows, M, lda = _operand(a, "a")
    rows_b, N, ldb = _operand(b, "b")
    if rows_b != rows:
        raise ValueError(f"a has {rows} rows, b {rows_b}")
    device = a.device
    if b.device != device:
        raise ValueError("all operands must be on the same device")
    E = _offsets(offsets, device)
    if c is None:
        with _allocating(stream, device):
            c = torch.empty((E, M, N), dtype=torch.float16, device=device)
    elif tuple(c.shape) != (E, M, N):
        raise ValueError(f"c has shape {tuple(c.shape)}, expected {(E, M, N)}")
    _, _, _, ldc, sc = _stacked(c, "c")
    if c.device != device:
        raise ValueError("all operands must be on the same device")
    args = (rows, E, M, N, a.data_ptr(), lda, b.data_ptr(), ldb, offsets.data_ptr(), c.data_ptr(), ldc, sc,
            _stream(stream, device))
    rc = (_call("expert_gemm_f16_tn", args, device, library) if cfg is None
          else _call("expert_gemm_f16_tn_cfg", (cfg, *args), device, library))
    if rc != TGEMM_OK:
        raise TgemmError(rc, "expert_gemm_f16_tn" if cfg is None else f"expert_gemm_f16_tn_cfg[{cfg}]")
    return c


def expert_gemm_select_config(form: str, rows, experts, M=0, N=0, K=0, A=256, lda=None, B=256, ldb=None,
                              stride_b=None) -> int:
    """The kernel (EXPERT_*) a product takes: ``form`` "nt" (trans_b), "nn" or "tn"; pointers are only
    looked at for null and alignment."""
    tn, nt = form == "tn", form == "nt"
    lda = max(1, M if tn else K) if lda is None else lda
    ldb = max(1, K if nt else N) if ldb is None else ldb
    stride_b = (0 if tn else N * K) if stride_b is None else stride_b
    return int(lib().expert_gemm_select_config(("nt", "nn", "tn").index(form), rows, experts, M, N, K, A, lda, B, ldb,
                                               stride_b))


def _once():
    import torch
    if torch.is_grad_enabled():
        raise RuntimeError("the expert functions have no second derivative (create_graph=True)")


def _like(*tensors):
    return tuple((t.shape, t.dtype, t.device) for t in tensors)


def _saved(ctx):
    """The saved tensors, checked to be what the forward pass saved (the library takes addresses):
    saved-tensor hooks may return others."""
    tensors = ctx.saved_tensors
    if _like(*tensors) != ctx.saved:
        raise RuntimeError("a saved-tensor hook returned another tensor than the forward pass saved")
    return tensors


def _ld(t):
    """Row stride of a 2-D tensor with contiguous rows, as the library takes it."""
    rows, cols = t.shape
    return t.stride(0) if rows > 1 else cols or 1


def _grad(t, name, shape, device):
    """An incoming gradient as the library takes it."""
    t = _row_major(t, name)
    if t.shape != shape or t.device != device:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)} on {device}")
    return t


def _ran(rc, name):
    if rc != TGEMM_OK:
        raise TgemmError(rc, name)


def autograd_functions():
    import torch
    f16 = torch.float16

    class ExpertGatherFunction(torch.autograd.Function):
        """(x, *plan) -> the sorted rows, those behind the last in use zero; dx[t] is the sum of its rows'
        gradients."""

        @staticmethod
        def forward(ctx, x, offsets, order, place):
            x = _row_major(x, "x")
            xs = expert_gather(x, ExpertOrder(offsets, order, place), zero_rest=True)
            ctx.save_for_backward(place)
            ctx.saved = _like(place)
            return xs

        @staticmethod
        def backward(ctx, dxs):
            _once()
            place = _saved(ctx)[0].contiguous()
            (T, k), device = place.shape, place.device
            H = dxs.shape[1]
            dxs = _grad(dxs, "dxs", (T * k, H), device)
            dx = torch.empty((T, H), dtype=f16, device=device)
            _ran(_call("expert_combine_f16", (T, k, T * k, H, dxs.data_ptr(), _ld(dxs), place.data_ptr(), None, DTYPE_F32,
                                              dx.data_ptr(), H or 1, _stream(None, device)), device), "expert_combine_f16")
            return dx, None, None, None

    class ExpertCombineFunction(torch.autograd.Function):
        """(y, weights or None, *plan) -> the tokens' weighted sums; gradients of the rows (zero behind the
        last one in use) and of the weights (zero for a slot of no expert)."""

        @staticmethod
        def forward(ctx, y, weights, offsets, order, place):
            y = _row_major(y, "y")
            weights = None if weights is None else weights.contiguous()
            out = expert_combine(y, ExpertOrder(offsets, order, place), weights)
            ctx.experts, ctx.rows = _offsets(offsets, y.device), y.shape
            # (y is read for the weights' gradient only)
            kept = (offsets, place) + (() if weights is None else (weights,)) + ((y,) if ctx.needs_input_grad[1] else ())
            ctx.save_for_backward(*kept)
            ctx.saved = _like(*kept)
            return out

        @staticmethod
        def backward(ctx, dout):
            _once()
            need_y, need_w = ctx.needs_input_grad[:2]
            offsets, place, *rest = (t.contiguous() for t in _saved(ctx))
            y, weights = rest.pop() if need_w else None, rest[0] if rest else None
            (T, k), (rows, H), device = place.shape, ctx.rows, place.device
            dout = _grad(dout, "dout", (T, H), device)
            dy = torch.empty((rows, H), dtype=f16, device=device) if need_y else None
            dw = torch.empty_like(weights) if need_w else None
            w, w_dtype = _weights(weights, (T, k), device)
            ld = H or 1
            _ran(_call("expert_combine_f16_backward",
                       (T, k, rows, H, dout.data_ptr(), _ld(dout), y.data_ptr() if need_w else None, ld, place.data_ptr(), w,
                        w_dtype, dy.data_ptr() if need_y else None, ld, dw.data_ptr() if need_w else None, offsets.data_ptr(),
                        ctx.experts, _stream(None, device)), device), "expert_combine_f16_backward")
            return dy, dw, None, None, None

    class ExpertGemmFunction(torch.autograd.Function):
        """c[p] = a[p] @ b[e]^T (no ReLU) for fp16 a (rows, K) and b (E, N, K), rows from offsets[E] on zero
        (offsets[0] is 0, as expert_sort writes it); da = dc b_e, db_e = dc_e^T a_e."""

        @staticmethod
        def forward(ctx, a, b, offsets):
            a = _row_major(a, "a")
            if b.dim() == 3 and b.numel() and (b.stride(2) != 1 or b.stride(1) < b.shape[2]):  # a broadcast weight
                b = b.contiguous()
            c = expert_gemm_f16(a, b, offsets, zero_rest=True)
            need_a, need_b, _ = ctx.needs_input_grad
            # (a is read for b's gradient and b for a's)
            kept = (offsets,) + ((b,) if need_a else ()) + ((a,) if need_b else ())
            ctx.save_for_backward(*kept)
            ctx.saved = _like(*kept)
            ctx.shapes = a.shape, b.shape
            return c

        @staticmethod
        def backward(ctx, dc):
            _once()
            need_a, need_b, _ = ctx.needs_input_grad
            offsets, *operands = _saved(ctx)
            offsets = offsets.contiguous()
            (rows, K), (E, N, _) = ctx.shapes
            device = offsets.device
            dc = _grad(dc, "dc", (rows, N), device)
            da = db = None
            stream = _stream(None, device)
            if need_a:
                b = operands[0]
                if b.stride(-1) != 1 or b.stride(1) < K:
                    b = b.contiguous()
                da = torch.empty((rows, K), dtype=f16, device=device)
                _ran(_call("expert_gemm_f16", (0, rows, E, K, N, dc.data_ptr(), _ld(dc), offsets.data_ptr(), b.data_ptr(),
                                               b.stride(1) if N > 1 else K or 1, b.stride(0) if E > 1 else 0, da.data_ptr(),
                                               K or 1, 0, 1, stream), device), "expert_gemm_f16")
            if need_b:
                a = _row_major(operands[-1], "a")
                db = torch.empty((E, N, K), dtype=f16, device=device)
                _ran(_call("expert_gemm_f16_tn", (rows, E, N, K, dc.data_ptr(), _ld(dc), a.data_ptr(), _ld(a),
                                                  offsets.data_ptr(), db.data_ptr(), K or 1, N * (K or 1), stream), device),
                     "expert_gemm_f16_tn")
            return da, db, None

    return {"ExpertGatherFunction": ExpertGatherFunction, "ExpertCombineFunction": ExpertCombineFunction,
            "ExpertGemmFunction": ExpertGemmFunction}
