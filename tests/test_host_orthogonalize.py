"""The orthogonalisation's entry points on the CPU: workspace sizes and refusals (every call
here returns before any HIP call)."""
import pytest

import tiled_dense_gemm_04_amd as tg

A16 = 256
BIG = 1 << 50


def call(batch=2, R=8, C=16, dtype=0, G=A16, ldg=16, sg=128, X=A16, ldx=16, sx=128, steps=5, ws=A16, nbytes=BIG):
    if nbytes == "short":
        nbytes = tg.orthogonalize_workspace_bytes(batch, R, C) - 1
    return tg.lib().orthogonalize_f16(batch, R, C, dtype, G, ldg, sg, X, ldx, sx, steps, 3.4445, -4.775, 2.0315, 1.0,
                                      ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), tg.TGEMM_EINVAL_DIM), (dict(R=-1), tg.TGEMM_EINVAL_DIM), (dict(C=1 << 31, ldg=1 << 31, ldx=1 << 31), tg.TGEMM_EINVAL_DIM),
    (dict(R=40000, C=40000, ldg=40000, ldx=40000), tg.TGEMM_EINVAL_DIM), (dict(C=tg.FAST_MAX_LD + 1, ldg=BIG, ldx=BIG), tg.TGEMM_EINVAL_DIM),
    (dict(steps=0), tg.TGEMM_EINVAL_DIM), (dict(steps=65), tg.TGEMM_EINVAL_DIM), (dict(dtype=2), tg.TGEMM_EINVAL_DIM),
    (dict(dtype=-1), tg.TGEMM_EINVAL_DIM),
    (dict(ldg=15), tg.TGEMM_EINVAL_LD), (dict(ldx=15), tg.TGEMM_EINVAL_LD), (dict(sg=-1), tg.TGEMM_EINVAL_LD),
    (dict(sx=127), tg.TGEMM_EINVAL_LD), (dict(sx=0), tg.TGEMM_EINVAL_LD),
    (dict(G=None), tg.TGEMM_ENULL), (dict(X=None), tg.TGEMM_ENULL), (dict(ws=None), tg.TGEMM_ENULL),
    (dict(G=A16 + 1), tg.TGEMM_EALIGN), (dict(G=A16 + 2, dtype=1), tg.TGEMM_EALIGN), (dict(X=A16 + 1), tg.TGEMM_EALIGN),
    (dict(ws=A16 + 128), tg.TGEMM_EALIGN), (dict(nbytes=1000), tg.TGEMM_EWORKSPACE),
    (dict(nbytes="short"), tg.TGEMM_EWORKSPACE),
    (dict(batch=0, G=None), tg.TGEMM_OK), (dict(R=0, X=None), tg.TGEMM_OK), (dict(C=0, ws=None), tg.TGEMM_OK),
])
def test_refusals(kw, code):
    assert call(**kw) == code


def test_workspace_bytes():
    ws = tg.orthogonalize_workspace_bytes
    assert ws(0, 5, 5) == 0 and ws(3, 0, 5) == 0
    assert ws(1, 100, 30) == ws(1, 30, 100) and ws(1, 64, 128) == ws(1, 1, 65)
    m, n = 4096, 16384
    assert ws(1, m, n) >= 8 * m * n + 4 * m * m + 8 * m
    assert 2.9 * ws(1, m, n) < ws(3, m, n) < 3.1 * ws(1, m, n)
    for bad in ((-1, 4, 4), (1, 1 << 31, 4), (1, 40000, 40000)):
        with pytest.raises(tg.TgemmError):
            ws(*bad)


def test_python_refusals():
    import torch
    with pytest.raises(ValueError, match="device tensor"):
        tg.orthogonalize(torch.zeros(4, 4, dtype=torch.float16))
    with pytest.raises(TypeError):
        tg.orthogonalize(torch.zeros(4, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="2-D"):
        tg.orthogonalize(torch.zeros(4, dtype=torch.float16))


def test_batch_limits():
    """Fewer than 2^32 threads in a launch: 512 per 4096 padded values, and the batch itself."""
    assert tg.orthogonalize_workspace_bytes((1 << 22) - 1, 8, 8) > 0
    for bad in ((1 << 22, 8, 8), (1 << 21, 256, 256)):
        with pytest.raises(tg.TgemmError) as e:
            tg.orthogonalize_workspace_bytes(*bad)
        assert e.value.code == tg.TGEMM_EINVAL_DIM
