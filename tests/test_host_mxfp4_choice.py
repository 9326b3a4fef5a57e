"""The kernel that an MXFP4 product of the package's wrappers ends up on, on the CPU: the call that
reaches the library is caught and its choice asked for."""
import pytest
import torch

import tiled_dense_gemm_04_amd as tg
from tiled_dense_gemm_04_amd import mxfp4


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
