"""The expert layer's entry points on the CPU: refusals, workspace sizes, kernel choice, and the
references' own checks (every library call here returns before any HIP call)."""
import os
import re

import numpy as np
import pytest

import expert_reference as ref
import tiled_dense_gemm_04_amd as tg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 256  # stands for an aligned device pointer; never dereferenced
DIM, LD, NULL, ALIGN, OK = tg.TGEMM_EINVAL_DIM, tg.TGEMM_EINVAL_LD, tg.TGEMM_ENULL, tg.TGEMM_EALIGN, tg.TGEMM_OK


def sort(T=10, k=2, E=8, ids=P, ldi=2, t=0, off=P, order=P, place=P, ws=None, nws=0):
    return tg.lib().expert_sort(T, k, E, ids, ldi, t, off, order, place, ws, nws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), DIM), (dict(k=-1), DIM), (dict(E=0), DIM), (dict(E=tg.MAX_EXPERTS + 1), DIM), (dict(t=2), DIM),
    (dict(T=tg.MAX_SLOTS, k=2), DIM), (dict(ldi=1), LD), (dict(ids=None), NULL), (dict(off=None), NULL), (dict(order=None), NULL),
    (dict(place=None), NULL), (dict(T=40000), NULL), (dict(T=40000, ws=P + 4, nws=1 << 20), ALIGN),
    (dict(T=40000, ws=P, nws=256 * 9 * 4 - 1), tg.TGEMM_EWORKSPACE), (dict(ids=P + 2), ALIGN), (dict(ids=P + 4, t=1), ALIGN),
    (dict(off=P + 2), ALIGN), (dict(T=0, off=None), NULL),
])
def test_sort_refusals(kw, code):
    assert sort(**kw) == code


def test_sort_workspace_bytes():
    f = tg.lib().expert_sort_workspace_bytes
    assert f(4096, 2, 8) == 0 and f(8193, 1, 8) == 256 * 9 * 4 and f(0, 0, 1) == 0
    assert f(-1, 1, 8) == DIM and f(1, 1, 0) == DIM and f(tg.MAX_SLOTS + 1, 1, 8) == DIM


def gather(T=10, k=2, rows=20, H=64, X=P, ldx=64, place=P, XS=P, ldxs=64, off=None, E=0):
    return tg.lib().expert_gather_f16(T, k, rows, H, X, ldx, place, XS, ldxs, off, E, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), DIM), (dict(rows=-1), DIM), (dict(H=1 << 31), DIM), (dict(T=1 << 20, H=1 << 16, ldx=1 << 16, ldxs=1 << 16), DIM),
    (dict(off=P, E=0), DIM), (dict(off=P, E=1025), DIM), (dict(ldx=63), LD), (dict(ldxs=63), LD), (dict(X=None), NULL),
    (dict(place=None), NULL), (dict(XS=None), NULL), (dict(X=P + 1), ALIGN), (dict(XS=P + 1), ALIGN), (dict(place=P + 2), ALIGN),
    (dict(off=P + 1, E=4), ALIGN), (dict(rows=0, XS=None), OK), (dict(H=0), OK), (dict(T=0, X=None), OK),
])
def test_gather_refusals(kw, code):
    assert gather(**kw) == code


def combine(T=10, k=2, rows=20, H=64, Y=P, ldy=64, place=P, w=P, wt=1, out=P, ldo=64):
    return tg.lib().expert_combine_f16(T, k, rows, H, Y, ldy, place, w, wt, out, ldo, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), DIM), (dict(H=-1), DIM), (dict(wt=2), DIM), (dict(ldy=63), LD), (dict(ldo=63), LD), (dict(Y=None), NULL),
    (dict(place=None), NULL), (dict(out=None), NULL), (dict(Y=P + 1), ALIGN), (dict(w=P + 2), ALIGN), (dict(w=P + 1, wt=0), ALIGN),
    (dict(T=0, out=None), OK), (dict(H=0), OK),
])
def test_combine_refusals(kw, code):
    assert combine(**kw) == code


def grad(T=10, k=2, rows=20, H=64, dO=P, lddo=64, Y=P, ldy=64, place=P, w=P, wt=1, dY=P, lddy=64, dw=P, off=None, E=0):
    return tg.lib().expert_combine_f16_backward(T, k, rows, H, dO, lddo, Y, ldy, place, w, wt, dY, lddy, dw, off, E, None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=-1), DIM), (dict(wt=-1), DIM), (dict(off=P, E=0), DIM), (dict(lddo=63), LD), (dict(ldy=63), LD), (dict(lddy=63), LD),
    (dict(dO=None), NULL), (dict(Y=None), NULL), (dict(place=None), NULL), (dict(dY=None, dw=None), NULL), (dict(dw=P + 2), ALIGN),
    (dict(dY=P + 1), ALIGN), (dict(T=0, dO=None), OK),
])
def test_combine_gradient_refusals(kw, code):
    assert grad(**kw) == code


def gemm(tb=1, rows=100, E=4, N=64, K=32, A=P, lda=32, off=P, B=P, ldb=32, sb=2048, C=P, ldc=64, cfg=None):
    args = (tb, rows, E, N, K, A, lda, off, B, ldb, sb, C, ldc, 0, 0, None)
    return tg.lib().expert_gemm_f16(*args) if cfg is None else tg.lib().expert_gemm_f16_cfg(cfg, *args)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), DIM), (dict(E=0), DIM), (dict(E=1025), DIM), (dict(N=1 << 31), DIM), (dict(K=-1), DIM),
    (dict(lda=31), LD), (dict(ldb=31), LD), (dict(tb=0, ldb=63), LD), (dict(ldc=63), LD), (dict(sb=-1), LD),
    (dict(A=None), NULL), (dict(B=None), NULL), (dict(C=None), NULL), (dict(off=None), NULL), (dict(A=P + 1), ALIGN),
    (dict(off=P + 2), ALIGN), (dict(rows=(1 << 31) - 1, N=65536, ldc=65536, sb=1 << 21), DIM),
    (dict(cfg=6), tg.TGEMM_EINVAL_CFG), (dict(cfg=-1), tg.TGEMM_EINVAL_CFG), (dict(cfg=2, A=P + 2), tg.TGEMM_EINVAL_CFG),
    (dict(cfg=1, lda=33), tg.TGEMM_EINVAL_CFG), (dict(cfg=3, sb=2049), tg.TGEMM_EINVAL_CFG),
    (dict(cfg=1, K=0), tg.TGEMM_EINVAL_CFG), (dict(rows=0, A=None), OK), (dict(N=0), OK),
])
def test_product_refusals(kw, code):
    assert gemm(**kw) == code


def gemm_tn(rows=100, E=4, M=64, N=32, A=P, lda=64, B=P, ldb=32, off=P, C=P, ldc=32, sc=2048, cfg=None):
    args = (rows, E, M, N, A, lda, B, ldb, off, C, ldc, sc, None)
    return tg.lib().expert_gemm_f16_tn(*args) if cfg is None else tg.lib().expert_gemm_f16_tn_cfg(cfg, *args)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), DIM), (dict(E=0), DIM), (dict(lda=63), LD), (dict(ldb=31), LD), (dict(ldc=31), LD), (dict(sc=2047), LD),
    (dict(A=None), NULL), (dict(C=None), NULL), (dict(off=None), NULL), (dict(C=P + 1), ALIGN),
    (dict(M=1 << 22, N=1 << 22, lda=1 << 22, ldb=1 << 22, ldc=1 << 22, sc=1 << 50), DIM), (dict(cfg=tg.EXPERT_32), tg.TGEMM_EINVAL_CFG), (dict(cfg=tg.EXPERT_64), tg.TGEMM_EINVAL_CFG),
    (dict(cfg=tg.EXPERT_128, M=63), tg.TGEMM_EINVAL_CFG), (dict(M=0), OK), (dict(N=0), OK),
])
def test_weight_product_refusals(kw, code):
    assert gemm_tn(**kw) == code


def test_kernel_choice():
    f = tg.expert_gemm_select_config
    for form in ("nt", "nn"):
        assert f(form, 64, 64, N=2048, K=4096) == tg.EXPERT_32
        assert f(form, 1, 64, N=2048, K=4096) == tg.EXPERT_32
        assert f(form, 16384, 16, N=4096, K=2048) == tg.EXPERT_TILES
        assert f(form, 1600, 16, N=512, K=512) == tg.EXPERT_TILES and f(form, 96, 16, N=512, K=512) == tg.EXPERT_32
        assert f(form, 784, 16, N=2048, K=512) == tg.EXPERT_64 and f(form, 783, 16, N=2048, K=512) == tg.EXPERT_32
        assert f(form, 784, 16, N=1024, K=512) == tg.EXPERT_TILES and f(form, 784, 16, N=1032, K=512) == tg.EXPERT_64
        assert f(form, 64, 8, N=64, K=63) == tg.EXPERT_GENERIC      # K is contiguous in A
        assert f(form, 64, 8, N=64, K=64, A=P + 2) == tg.EXPERT_GENERIC
        assert f(form, 64, 8, N=64, K=64, stride_b=4097) == tg.EXPERT_GENERIC
        assert f(form, 64, 8, N=64, K=0) == tg.EXPERT_GENERIC
        assert f(form, 0, 8, N=64, K=64) == -100 and f(form, 64, 0, N=64, K=64) == DIM
    assert f("nt", 64, 8, N=65, K=64) == tg.EXPERT_32 and f("nn", 64, 8, N=65, K=64) == tg.EXPERT_GENERIC
    assert f("tn", 8192, 8, M=2048, N=2048) == tg.EXPERT_TILES and f("tn", 1, 8, M=256, N=256) == tg.EXPERT_TILES
    assert f("tn", 8192, 8, M=255, N=256) == tg.EXPERT_GENERIC


def test_header_limits():
    text = open(os.path.join(ROOT, "include", "tgemm_ops.h")).read()
    assert f"#define TGEMM_MAX_EXPERTS {tg.MAX_EXPERTS}" in text and "(((int64_t)1 << 26) - 1024)" in text
    for name, value in (("GENERIC", tg.EXPERT_GENERIC), ("32", tg.EXPERT_32), ("128", tg.EXPERT_128), ("256", tg.EXPERT_256),
                        ("TILES", tg.EXPERT_TILES), ("64", tg.EXPERT_64)):
        assert re.search(rf"#define TGEMM_EXPERT_{name} {value}\b", text)


def test_python_refusals():
    import torch
    ids = torch.zeros((4, 2), dtype=torch.int64)
    with pytest.raises(ValueError, match="device tensor"):
        tg.expert_sort(ids, 8)
    with pytest.raises(TypeError, match="int32 or int64"):
        tg.expert_sort(ids.float(), 8)
    with pytest.raises(ValueError, match="2-D"):
        tg.expert_sort(ids[0], 8)
    x = torch.zeros((4, 64), dtype=torch.float16)
    plan = tg.ExpertOrder(*(torch.zeros(s, dtype=torch.int32) for s in ((9,), (8,), (4, 2))))
    with pytest.raises(ValueError, match="device tensor"):
        tg.expert_gather(x, plan)
    with pytest.raises(TypeError, match="float16"):
        tg.expert_combine(x.float(), plan)
    with pytest.raises(ValueError, match="device tensor"):
        tg.expert_gemm_f16(x, torch.zeros((8, 32, 64), dtype=torch.float16), plan.offsets)
    with pytest.raises(TypeError, match="float16"):
        tg.expert_gemm_f16_tn(x.double(), x, plan.offsets)


def test_reference_sort_is_stable_and_drops():
    ids = np.array([[2, 0], [-1, 2], [0, 9], [2, 1]])
    offsets, order, place = ref.sort(ids, 3)
    assert offsets.tolist() == [0, 2, 3, 6] and order.tolist() == [1, 4, 7, 0, 3, 6, -1, -1]
    assert place.tolist() == [[3, 0], [-1, 4], [1, -1], [5, 2]]


def test_reference_bound_sees_a_dropped_term():
    """The exact operands tell a product with one term left out; the bound on normal ones does at these sizes."""
    rng = np.random.default_rng(0)
    a, b = rng.standard_normal((4, 64)), rng.standard_normal((1, 8, 64))
    want, size = ref.products(a, b, [0, 4], True, np.zeros((4, 8)))
    less, _ = ref.products(a[:, :63], b[:, :, :63], [0, 4], True, np.zeros((4, 8)))
    assert (np.abs(less - want) > ref.product_bound(want, size, 64)).mean() > 0.5
