"""The MXFP4 entry points on the CPU: exported symbols, refusals and kernel choice (every call
here returns before any HIP call)."""
import os
import re
import subprocess
import sys

import pytest

import tiled_dense_gemm_04_amd as tg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A16 = 256  # stands for an aligned device pointer; never dereferenced


def header():
    return open(os.path.join(ROOT, "include", "tgemm_ops.h")).read()


def test_header_symbols_are_exported():
    syms = sorted(set(re.findall(r"^TGEMM_API\s+[\w\s\*]*?\b(\w+)\s*\(", header(), re.M)))
    assert sorted(tg.OPS_EXPORTS) == syms
    for path in (tg.LIBRARY, tg.STAMPS_LIBRARY, tg.DEBUGFILL_LIBRARY):
        out = subprocess.run(["nm", "-D", "--defined-only", path], capture_output=True, text=True, check=True).stdout
        names = {ln.split()[-1] for ln in out.splitlines() if ln.strip()}
        assert set(syms) <= names


def test_constants_match_header():
    text = header()
    for name, value in (("GENERIC", tg.MX_GENERIC), ("SKINNY", tg.MX_SKINNY), ("128", tg.MX_128), ("256", tg.MX_256), ("64", tg.MX_64)):
        assert re.search(rf"#define TGEMM_MX_{name} {value}\b", text)
    assert "(TGEMM_MAX_DIM - 512)" in text and tg.MX_MAX_DIM == (1 << 31) - 512


def quant(R=8, K=64, X=A16, ldx=64, Q=A16, ldq=32, S=A16, lds=16, QT=None, ldqt=0, ST=None, ldst=0):
    return tg.lib().mxfp4_quant(R, K, X, ldx, Q, ldq, S, lds, QT, ldqt, ST, ldst, None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), tg.TGEMM_EINVAL_DIM), (dict(K=tg.MX_MAX_DIM + 1, ldx=1 << 40), tg.TGEMM_EINVAL_DIM),
    (dict(ldx=63), tg.TGEMM_EINVAL_LD), (dict(ldq=31), tg.TGEMM_EINVAL_LD), (dict(lds=1), tg.TGEMM_EINVAL_LD),
    (dict(K=33, lds=1), tg.TGEMM_EINVAL_LD), (dict(K=33, ldq=31), tg.TGEMM_EINVAL_LD),
    (dict(X=None), tg.TGEMM_ENULL), (dict(Q=None), tg.TGEMM_ENULL), (dict(S=None), tg.TGEMM_ENULL),
    (dict(Q=None, S=None), tg.TGEMM_ENULL), (dict(QT=A16, ldqt=16, ldst=1), tg.TGEMM_ENULL),
    (dict(QT=A16, ST=A16, ldqt=15, ldst=1), tg.TGEMM_EINVAL_LD), (dict(QT=A16, ST=A16, ldqt=16, ldst=0), tg.TGEMM_EINVAL_LD),
    (dict(X=A16 + 1), tg.TGEMM_EALIGN),
    (dict(R=1 << 28, K=1 << 10, ldx=1 << 10, ldq=512, lds=32), tg.TGEMM_EINVAL_DIM),
    (dict(R=0, X=None), tg.TGEMM_OK), (dict(K=0, ldq=16, X=None), tg.TGEMM_OK),
])
def test_quant_refusals(kw, code):
    assert quant(**kw) == code


def dequant(R=8, K=64, Q=A16, ldq=32, S=A16, lds=2, X=A16, ldx=64):
    return tg.lib().mxfp4_dequant(R, K, Q, ldq, S, lds, X, ldx, None)


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), tg.TGEMM_EINVAL_DIM), (dict(K=-3), tg.TGEMM_EINVAL_DIM), (dict(ldx=63), tg.TGEMM_EINVAL_LD),
    (dict(ldq=16), tg.TGEMM_EINVAL_LD), (dict(lds=1), tg.TGEMM_EINVAL_LD), (dict(Q=None), tg.TGEMM_ENULL),
    (dict(S=None), tg.TGEMM_ENULL), (dict(X=None), tg.TGEMM_ENULL), (dict(X=A16 + 1), tg.TGEMM_EALIGN),
    (dict(R=0, Q=None), tg.TGEMM_OK), (dict(R=1 << 28, K=1 << 10, ldx=1 << 10, ldq=512, lds=32), tg.TGEMM_EINVAL_DIM),
])
def test_dequant_refusals(kw, code):
    assert dequant(**kw) == code


def gemm(M=8, N=8, K=64, A=A16, lda=32, SA=A16, ldsa=16, B=A16, ldb=32, SB=A16, ldsb=16, C=A16, ldc=8, cfg=None):
    args = (M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc, 0, None)
    return tg.lib().mxfp4_gemm(*args) if cfg is None else tg.lib().mxfp4_gemm_cfg(cfg, *args)


def gemm_f16(M=8, N=8, K=64, A=A16, lda=64, B=A16, ldb=32, SB=A16, ldsb=16, C=A16, ldc=8, cfg=None):
    args = (M, N, K, A, lda, B, ldb, SB, ldsb, C, ldc, 0, None)
    return tg.lib().mxfp4_gemm_f16(*args) if cfg is None else tg.lib().mxfp4_gemm_f16_cfg(cfg, *args)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), tg.TGEMM_EINVAL_DIM), (dict(N=tg.MX_MAX_DIM + 1, ldc=1 << 40), tg.TGEMM_EINVAL_DIM),
    (dict(lda=31), tg.TGEMM_EINVAL_LD), (dict(ldb=31), tg.TGEMM_EINVAL_LD), (dict(ldsb=1), tg.TGEMM_EINVAL_LD),
    (dict(ldc=7), tg.TGEMM_EINVAL_LD), (dict(A=None), tg.TGEMM_ENULL), (dict(B=None), tg.TGEMM_ENULL),
    (dict(SB=None), tg.TGEMM_ENULL), (dict(C=None), tg.TGEMM_ENULL), (dict(C=A16 + 1), tg.TGEMM_EALIGN),
    (dict(cfg=-1), tg.TGEMM_EINVAL_CFG), (dict(cfg=5), tg.TGEMM_EINVAL_CFG),
    (dict(cfg=tg.MX_SKINNY, M=tg.MX_SKINNY_ROWS + 1), tg.TGEMM_EINVAL_CFG), (dict(cfg=tg.MX_256, B=A16 + 4), tg.TGEMM_EINVAL_CFG),
    (dict(cfg=tg.MX_128, ldb=40), tg.TGEMM_EINVAL_CFG),
    (dict(M=0, A=None), tg.TGEMM_OK), (dict(N=0, B=None, C=None), tg.TGEMM_OK),
    (dict(M=1 << 30, N=1 << 30, ldc=1 << 30), tg.TGEMM_EINVAL_DIM),
])
def test_gemm_refusals(kw, code):
    assert gemm(**kw) == code
    if "lda" not in kw:
        assert gemm_f16(**kw) == code


def test_gemm_more_refusals():
    assert gemm(ldsa=1) == tg.TGEMM_EINVAL_LD
    assert gemm(SA=None) == tg.TGEMM_ENULL
    assert gemm_f16(lda=63) == tg.TGEMM_EINVAL_LD
    assert gemm_f16(A=A16 + 1) == tg.TGEMM_EALIGN
    assert gemm_f16(cfg=tg.MX_64) == tg.TGEMM_EINVAL_CFG
    assert gemm_f16(cfg=tg.MX_128, lda=65) == tg.TGEMM_EINVAL_CFG
    assert gemm_f16(cfg=tg.MX_256, A=A16 + 2) == tg.TGEMM_EINVAL_CFG
    assert gemm_f16(cfg=tg.MX_SKINNY, B=A16 + 8) == tg.TGEMM_EINVAL_CFG


def test_kernel_choice():
    sel = tg.mxfp4_select_config
    for f16 in (False, True):
        assert sel(0, 8, 64, f16) == tg.SELECT_NOOP and sel(8, 8, 0, f16) == tg.SELECT_ZERO_FILL
        assert sel(1, 4096, 4096, f16) == tg.MX_SKINNY
        assert sel(8192, 8192, 8192, f16) == tg.MX_256
        assert sel(2048, 1024, 4096, f16) == (tg.MX_128 if f16 else tg.MX_64)
        assert sel(64, 4096, 4096, f16) == tg.MX_SKINNY
        assert sel(128, 2048, 96, f16) == (tg.MX_SKINNY if f16 else tg.MX_64)
        assert sel(2048, 2048, 4096, f16) == tg.MX_128
        # any N, and scales or codes the copies cannot take
        assert sel(4095, 4097, 64, f16) == tg.MX_256
        assert sel(300, 300, 96, f16, ldsb=3) == tg.MX_GENERIC
        assert sel(300, 300, 96, f16, B=A16 + 8) == tg.MX_GENERIC
        assert sel(300, 300, 96, f16, SB=A16 + 4) == tg.MX_GENERIC
        assert sel(300, 300, 96, f16, ldb=2 * tg.FAST_MAX_LD + 16) == tg.MX_GENERIC
    assert sel(300, 300, 96, False, ldsa=3) == tg.MX_GENERIC
    assert sel(300, 300, 96, False, SA=A16 + 1) == tg.MX_GENERIC
    assert sel(300, 300, 100, True) == tg.MX_GENERIC      # K no multiple of 8
    assert sel(100, 300, 101, True, A=A16 + 2, lda=107) == tg.MX_SKINNY
    assert sel(300, 300, 96, True, lda=100) == tg.MX_GENERIC
    assert sel(300, 300, 96, True, A=A16 + 2) == tg.MX_GENERIC
    assert sel(300, 300, 100, False) == tg.MX_64         # codes are whole blocks: any K


def test_python_refusals():
    import torch
    x = torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="device tensor"):
        tg.mxfp4_quant(x)
    with pytest.raises(TypeError):
        tg.mxfp4_quant(x.float())
    q, s = tg.mxfp4_empty(4, 70, "cpu")
    assert q.shape == (4, 48) and s.shape == (4, 3) and s.stride(0) == 16
    with pytest.raises(ValueError, match="device tensor"):
        tg.mxfp4_gemm(q, s, q, s)
    with pytest.raises(TypeError):
        tg.mxfp4_dequant(q.float(), s, 70)


def test_launch_limits():
    """Fewer than 2^32 threads in a launch: 128 blocks per workgroup of 256 threads, 16 rows of
    the weight per skinny workgroup of up to 1024, tiles of 512 threads."""
    most = (1 << 31) - 128   # blocks
    assert quant(R=1 << 26, K=1024, ldx=1024, ldq=512, lds=32) == tg.TGEMM_EINVAL_DIM
    assert dequant(R=1 << 26, K=1024, ldx=1024, ldq=512, lds=32) == tg.TGEMM_EINVAL_DIM
    assert (1 << 26) * 32 > most
    wide = 16 * ((1 << 22) - 1)   # columns of the skinny kernel
    for f16 in (False, True):
        assert tg.mxfp4_select_config(1, wide, 32, f16) == tg.MX_SKINNY
        assert tg.mxfp4_select_config(1, wide + 1, 32, f16) not in (tg.MX_SKINNY, tg.MX_GENERIC)
    for product in (gemm, gemm_f16):
        assert product(N=wide + 1, ldc=wide + 1, cfg=tg.MX_SKINNY) == tg.TGEMM_EINVAL_CFG
        # 2^24 tiles of 128 x 128
        assert product(M=33, N=(1 << 31) - 1024, ldc=1 << 31, cfg=tg.MX_128) == tg.TGEMM_EINVAL_DIM


def test_library_before_torch():
    """A program that asks the library for a size or a choice before it imports torch has one HIP
    runtime in the process: torch's own."""
    code = ("import tiled_dense_gemm_04_amd as tg\n"
            "assert tg.orthogonalize_workspace_bytes(1, 64, 64) > 0\n"
            "import torch\n"
            "maps = {l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}\n"
            "assert len(maps) == 1, maps\n")
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)
