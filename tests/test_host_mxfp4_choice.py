"""The kernel that an MXFP4 product of the package's wrappers ends up on, on the CPU: the call that
reaches the library is caught and its choice asked for."""
import pytest
import torch

import tiled_dense_gemm_04_amd as tg
from tiled_dense_gemm_04_amd import mxfp4

A16 = 256  # stands for an aligned device pointer; never dereferenced


@pytest.fixture
def launched(monkeypatch):
    """Calls on CPU tensors, caught before the library: [(entry point, arguments)]."""
    calls = []

    def operand(t, name):
        rows, cols = t.shape
        return rows, cols, t.stride(0) if rows > 1 else max(1, cols)

    matrix = mxfp4._matrix

    class OnDevice(torch.Tensor):
        is_cuda = True

    monkeypatch.setattr(mxfp4, "_operand", operand)
    monkeypatch.setattr(mxfp4, "_matrix", lambda codes, scale, name: matrix(codes.as_subclass(OnDevice), scale.as_subclass(OnDevice), name))
    monkeypatch.setattr(mxfp4, "_stream", lambda stream, device: 0)
    monkeypatch.setattr(mxfp4, "_call", lambda name, args, device, library=None: calls.append((name, args)) or tg.TGEMM_OK)
    return calls


def choice_f16(args):
    M, N, K, A, lda, B, ldb, SB, ldsb, C, ldc = args[:11]
    return tg.mxfp4_select_config(M, N, K, True, A=A, lda=lda, B=B, ldb=ldb, SB=SB, ldsb=ldsb, C=C, ldc=ldc)


def rows(M, K, off=0, ld=None):
    """(M, K) fp16 at `off` elements from a 16-byte boundary, rows `ld` apart."""
    ld = K if ld is None else ld
    buf = torch.zeros(off + M * ld + 8, dtype=torch.float16)
    at = (-buf.data_ptr() // 2) % 8 + off
    return buf[at:].as_strided((M, K), (ld, 1))


# Around each limit of the skinny kernel's choice, in rows and in width
SIZES = [(1, 4096), (32, 40000), (33, 12288), (33, 12304), (64, 20000), (65, 8192), (100, 8192), (128, 8000), (200, 8192),
         (256, 4096), (256, 8192), (257, 300), (300, 300), (1000, 2000)]


@pytest.mark.parametrize("M,N", SIZES)
def test_odd_rows_of_a_leave_the_generic_kernel(launched, M, N):
    for K, off, ld in ((1001, 0, None), (1000, 1, None), (1000, 0, 1003), (4095, 3, 4100), (40, 4, None)):
        kb = -(-K // 32)
        codes, scale = mxfp4.mxfp4_empty(N, K, "cpu")
        mxfp4.mxfp4_gemm_f16(rows(M, K, off, ld), codes, scale, c=torch.empty(M, N, dtype=torch.float16))
        name, args = launched.pop()
        assert name == "mxfp4_gemm_f16" and args[0] == M and args[1] == N and -(-args[2] // 32) == kb
        assert choice_f16(args) != tg.MX_GENERIC, (M, N, K, off, ld)
        # what the tiles get is the choice of padded rows
        whole = tg.mxfp4_select_config(M, N, -(-K // 8) * 8, True)
        assert choice_f16(args) == whole, (M, N, K, off, ld)


def test_no_copy_where_it_would_not_help(launched):
    a = rows(100, 1001)
    for codes, scale in ((torch.zeros(8192, 512 + 16, dtype=torch.uint8)[:, 4:516], torch.zeros(8192, 32, dtype=torch.uint8)),
                         mxfp4.mxfp4_empty(300, 1001, "cpu")):
        mxfp4.mxfp4_gemm_f16(a, codes, scale, c=torch.empty(100, codes.shape[0], dtype=torch.float16))
        assert launched.pop()[1][3] == a.data_ptr()


def test_choice_without_a_copy():
    """The C entry point for an A that the tiles cannot take: the skinny kernel up to 256 rows and four
    rounds of its workgroups, then the generic one (measured faster there)."""
    sel = tg.mxfp4_select_config
    for M, N, K in ((256, 4096, 3163), (128, 8000, 7611), (65, 8192, 2001), (100, 8192, 4095), (64, 16384, 1001)):
        assert sel(M, N, K, True) == tg.MX_SKINNY
        assert sel(M, N, -(-K // 8) * 8, True) == tg.MX_128
    for M, N, K in ((256, 4097, 3163), (200, 8192, 4095), (64, 16385, 1001), (257, 64, 1001)):
        assert sel(M, N, K, True) == tg.MX_GENERIC


def choice(args):
    M, N, K, A, lda, SA, ldsa, B, ldb, SB, ldsb, C, ldc = args[:13]
    return tg.mxfp4_select_config(M, N, K, False, A=A, lda=lda, SA=SA, ldsa=ldsa, B=B, ldb=ldb, SB=SB, ldsb=ldsb, C=C, ldc=ldc)


def close(R, K):
    """An MXFP4 matrix whose scales' rows lie close together, as a copy of a padded one has them."""
    codes, scale = mxfp4.mxfp4_empty(R, K, "cpu")
    return codes, scale.clone(memory_format=torch.contiguous_format)


@pytest.mark.parametrize("M,N", SIZES)
def test_close_scales_leave_the_generic_kernel(launched, M, N):
    for K in (1050, 2880):
        b = close(N, K)
        assert b[1].stride(0) == -(-K // 32) and b[1].stride(0) % 16
        out = torch.empty(M, N, dtype=torch.float16)
        mxfp4.mxfp4_gemm_f16(rows(M, K), *b, c=out)
        name, args = launched.pop()
        assert name == "mxfp4_gemm_f16" and choice_f16(args) == tg.mxfp4_select_config(M, N, -(-K // 8) * 8, True)
        for a in (close(M, K), mxfp4.mxfp4_empty(M, K, "cpu")):
            mxfp4.mxfp4_gemm(*a, *b, c=out)
            name, args = launched.pop()
            assert name == "mxfp4_gemm" and choice(args) == tg.mxfp4_select_config(M, N, K)


def test_small_products_take_close_scales_as_they_lie(launched):
    a, b = close(300, 100), close(300, 100)
    mxfp4.mxfp4_gemm(*a, *b, c=torch.empty(300, 300, dtype=torch.float16))
    args = launched.pop()[1]
    assert args[5] == a[1].data_ptr() and args[9] == b[1].data_ptr() and choice(args) == tg.MX_GENERIC


def test_choice_of_close_scales():
    """The C entry points: the skinny kernel takes scales of any stride and base, up to 4 rounds of its
    workgroups with binary16 A, 16 with MXFP4 A."""
    sel = tg.mxfp4_select_config
    for f16 in (False, True):
        for lds in (90, 91, 1000):
            assert sel(1, 8192, 2880, f16, ldsb=lds) == tg.MX_SKINNY
            assert sel(32, 40000, 2880, f16, ldsb=lds) == tg.MX_SKINNY
            assert sel(256, 4096, 2880, f16, ldsb=lds) == tg.MX_SKINNY
        assert sel(64, 4096, 2880, f16, SB=A16 + 3) == tg.MX_SKINNY
        assert sel(257, 4096, 2880, f16, ldsb=90) == tg.MX_GENERIC
    assert sel(16, 8192, 2880, ldsa=90) == sel(16, 8192, 2880, SA=A16 + 1) == tg.MX_SKINNY
    assert sel(256, 16384, 2880, ldsb=90) == tg.MX_SKINNY and sel(256, 16400, 2880, ldsb=90) == tg.MX_GENERIC
    assert sel(256, 4112, 2880, True, ldsb=90) == tg.MX_GENERIC
    assert sel(1, 8192, 2880, B=A16 + 8) == tg.MX_GENERIC


def test_forced_kernels_and_close_scales():
    """A forced tile kernel refuses scales that it cannot read."""
    for cfg in (tg.MX_128, tg.MX_256):
        for SB, ldsb in ((A16 + 1, 16), (A16, 9)):
            rc = tg.lib().mxfp4_gemm_f16_cfg(cfg, 8, 8, 256, A16, 256, A16, 128, SB, ldsb, A16, 8, 0, None)
            assert rc == tg.TGEMM_EINVAL_CFG
            rc = tg.lib().mxfp4_gemm_cfg(cfg, 8, 8, 256, A16, 128, A16, 16, A16, 128, SB, ldsb, A16, 8, 0, None)
            assert rc == tg.TGEMM_EINVAL_CFG
            rc = tg.lib().mxfp4_gemm_cfg(cfg, 8, 8, 256, A16, 128, SB, ldsb, A16, 128, A16, 16, A16, 8, 0, None)
            assert rc == tg.TGEMM_EINVAL_CFG
