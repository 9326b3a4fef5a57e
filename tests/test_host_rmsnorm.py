"""The norm's entry points on the CPU: refusals, workspace sizes and the reference's own pieces (every
library call here returns before any HIP call)."""
import os
import re

import numpy as np
import pytest

import norm_reference as ref
import tiled_dense_gemm_04_amd as tg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 256  # stands for an aligned device pointer; never dereferenced
F16, F32 = 0, 1


def norm(R=4, K=64, X=P, ldx=64, r=None, ldr=64, rt=F16, W=P, wt=F16, eps=1e-6, ro=None, ldro=64, Y=P, ldy=64, Q=None,
         ldq=64, s=None):
    return tg.lib().rmsnorm_f16(R, K, X, ldx, r, ldr, rt, W, wt, eps, ro, ldro, Y, ldy, Q, ldq, s, None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), tg.TGEMM_EINVAL_DIM), (dict(K=-1), tg.TGEMM_EINVAL_DIM), (dict(K=tg.NORM_MAX_K + 1, ldx=1 << 20), tg.TGEMM_EINVAL_DIM),
    (dict(R=1 << 31), tg.TGEMM_EINVAL_DIM), (dict(R=1 << 24, K=4096, ldx=4096, ldy=4096), tg.TGEMM_EINVAL_DIM),
    (dict(R=1 << 28), tg.TGEMM_EINVAL_DIM), (dict(wt=2), tg.TGEMM_EINVAL_DIM), (dict(r=P, rt=-1), tg.TGEMM_EINVAL_DIM),
    (dict(eps=-1.0), tg.TGEMM_EINVAL_DIM), (dict(eps=float("nan")), tg.TGEMM_EINVAL_DIM),
    (dict(ldx=63), tg.TGEMM_EINVAL_LD), (dict(ldy=63), tg.TGEMM_EINVAL_LD), (dict(r=P, ldr=63), tg.TGEMM_EINVAL_LD),
    (dict(r=P, ro=P, ldro=63), tg.TGEMM_EINVAL_LD), (dict(Q=P, s=P, ldq=63), tg.TGEMM_EINVAL_LD),
    (dict(X=None), tg.TGEMM_ENULL), (dict(W=None), tg.TGEMM_ENULL), (dict(Y=None), tg.TGEMM_ENULL),
    (dict(Q=P), tg.TGEMM_ENULL), (dict(s=P), tg.TGEMM_ENULL), (dict(ro=P), tg.TGEMM_ENULL),
    (dict(X=P + 1), tg.TGEMM_EALIGN), (dict(W=P + 2, wt=F32), tg.TGEMM_EALIGN), (dict(r=P + 2, rt=F32), tg.TGEMM_EALIGN),
    (dict(r=P, ro=P + 1), tg.TGEMM_EALIGN), (dict(Q=P + 1, s=P + 2), tg.TGEMM_EALIGN),
    (dict(R=0, X=None), tg.TGEMM_OK), (dict(K=0, X=None), tg.TGEMM_OK),
])
def test_refusals(kw, code):
    assert norm(**kw) == code


def backward(R=4, K=64, dY=P, lddy=64, H=P, ldh=64, ht=F16, W=P, wt=F16, eps=1e-6, dH=None, lddh=64, dX=P, lddx=64, dR=None,
             lddr=64, dW=P, ws=P, nws=1 << 20):
    return tg.lib().rmsnorm_f16_backward(R, K, dY, lddy, H, ldh, ht, W, wt, eps, dH, lddh, dX, lddx, dR, lddr, dW, ws, nws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), tg.TGEMM_EINVAL_DIM), (dict(K=tg.NORM_MAX_K + 1), tg.TGEMM_EINVAL_DIM), (dict(ht=2), tg.TGEMM_EINVAL_DIM),
    (dict(wt=-1), tg.TGEMM_EINVAL_DIM), (dict(lddy=63), tg.TGEMM_EINVAL_LD), (dict(ldh=1), tg.TGEMM_EINVAL_LD),
    (dict(lddx=63), tg.TGEMM_EINVAL_LD), (dict(dH=P, lddh=63), tg.TGEMM_EINVAL_LD), (dict(dR=P, lddr=63), tg.TGEMM_EINVAL_LD),
    (dict(dY=None), tg.TGEMM_ENULL), (dict(H=None), tg.TGEMM_ENULL), (dict(W=None), tg.TGEMM_ENULL),
    (dict(eps=-1.0), tg.TGEMM_EINVAL_DIM), (dict(dX=None), tg.TGEMM_ENULL), (dict(ws=None), tg.TGEMM_ENULL),
    (dict(ws=P + 4), tg.TGEMM_EALIGN), (dict(H=P + 2, ht=F32), tg.TGEMM_EALIGN), (dict(dW=P + 1), tg.TGEMM_EALIGN),
    (dict(dR=P + 2, ht=F32), tg.TGEMM_EALIGN), (dict(nws=2 * 64 * 4 - 1, R=33), tg.TGEMM_EWORKSPACE),
    (dict(K=0), tg.TGEMM_OK), (dict(R=0, dW=None), tg.TGEMM_OK),
])
def test_backward_refusals(kw, code):
    assert backward(**kw) == code


def test_workspace_bytes():
    f = tg.lib().rmsnorm_f16_backward_workspace_bytes
    assert f(0, 64) == 0 and f(5, 0) == 0 and f(-1, 64) == tg.TGEMM_EINVAL_DIM
    assert f(1, 64) == 64 * 4 and f(33, 64) == 2 * 64 * 4 and f(3, 4096) == 2 * 4096 * 4 and f(1 << 20, 4096) == f(1 << 19, 4096) > 0


def test_header_limits():
    text = open(os.path.join(ROOT, "include", "tgemm_ops.h")).read()
    assert re.search(rf"#define TGEMM_NORM_MAX_K {tg.NORM_MAX_K}\b", text)


def test_python_refusals():
    import torch
    x, w = torch.zeros((4, 64), dtype=torch.float16), torch.ones(64, dtype=torch.float16)
    with pytest.raises(ValueError, match="device tensor"):
        tg.rmsnorm(x, w)
    with pytest.raises(TypeError, match="float16"):
        tg.rmsnorm(x.float(), w)
    with pytest.raises(TypeError, match="torch.Tensor"):
        tg.rmsnorm_fp8_block([1.0], w)
    with pytest.raises(TypeError, match="device tensor"):
        tg.RmsNormFunction.apply(x, w, None, 1e-6)


def test_reference_e4m3():
    """The grid's rounding takes every code to itself and midpoints to the even neighbour."""
    codes = np.arange(127, dtype=np.uint8)
    v = ref.e4m3_value(codes)
    assert np.array_equal(ref.e4m3(v), v) and v[-1] == 448 and (np.diff(v) > 0).all()
    mid = (v[1:] + v[:-1]) / 2
    even = np.where(codes[1:] % 2 == 0, v[1:], v[:-1])
    assert np.array_equal(ref.e4m3(mid), even)


def test_reference_bound_holds_for_float32_and_not_for_less():
    """A float32 emulation of the sums stays inside y's bound; rounding y to 10 bits first does not."""
    rng = np.random.default_rng(0)
    h = rng.standard_normal((50, 1000)).astype(np.float16)
    w = (1 + 0.2 * rng.standard_normal(1000)).astype(np.float16)
    y, _ = ref.norm(h, w, 1e-6)
    f = h.astype(np.float32)
    rstd = (1 / np.sqrt((f * f).mean(1, dtype=np.float32) + np.float32(1e-6))).astype(np.float32)
    got = (f * rstd[:, None] * w.astype(np.float32)).astype(np.float16)
    assert (np.abs(got - y) <= ref.y_bound(y)).all()
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 1e-30))) - 9)
    assert (np.abs(np.round(y / step) * step - y) > ref.y_bound(y)).any()
