"""MXFP4 products of operands that lie otherwise than the package allocates them, at the sizes where
the kernels' ranges meet, against float64."""
import numpy as np
import pytest

import mx_reference as mx
from gpu_util import log, to_dev, torch_cuda

import tiled_dense_gemm_04_amd as tg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = torch_cuda()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tg.lib()
    return torch


def padded(codes, scale):
    """Device copies as the package lays them out, NaN scales in the padding."""
    s = np.full((len(scale), -(-scale.shape[1] // 16) * 16), 255, dtype=np.uint8)
    s[:, :scale.shape[1]] = scale
    return to_dev(codes), to_dev(s)[:, :scale.shape[1]]


# One side and the other of the skinny kernel's four rounds; wide enough for tiles at few rows
@pytest.mark.parametrize("M,N,K", [(33, 16400, 101), (65, 8192, 203), (100, 8192, 1001), (128, 8000, 331), (200, 8192, 101),
                                   (256, 4096, 203), (256, 8200, 77)])
def test_odd_rows_of_a(gpu, M, N, K):
    rng = np.random.default_rng(M + N)
    a = rng.standard_normal((M, K)).astype(np.float16)
    B, sb = mx.random_matrix(rng, N, K, 118, 126)
    b = padded(B, sb)
    ref, tol = mx.product(a.astype(np.float64), mx.values(B, sb)[:, :K])
    for off, ld in ((0, K), (1, K + 2), (8, K + 5)):
        buf = gpu.full((off + M * ld + 8,), float("nan"), dtype=gpu.float16, device="cuda")
        x = buf[off:].as_strided((M, K), (ld, 1))
        x.copy_(to_dev(a))
        side = gpu.cuda.Stream()
        side.wait_stream(gpu.cuda.current_stream())
        log(f"{M}x{N}x{K} at {off}, stride {ld}")
        out = gpu.full((M, N + 3), 5.0, dtype=gpu.float16, device="cuda")
        tg.mxfp4_gemm_f16(x, *b, c=out[:, :N])
        mx.check(out[:, :N].cpu().numpy(), ref, tol)
        assert (out[:, N:] == 5.0).all()
        other = tg.mxfp4_gemm_f16(x, *b, stream=side)
        side.synchronize()
        assert gpu.equal(other, out[:, :N])
        # through the C entry point no copy is made
        c = gpu.empty((M, N), dtype=gpu.float16, device="cuda")
        rc = tg.lib().mxfp4_gemm_f16(M, N, K, x.data_ptr(), ld, b[0].data_ptr(), b[0].stride(0), b[1].data_ptr(),
                                     b[1].stride(0), c.data_ptr(), N, 0, gpu.cuda.current_stream().cuda_stream)
        assert rc == tg.TGEMM_OK
        mx.check(c.cpu().numpy(), ref, tol)
