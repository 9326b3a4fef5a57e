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


def close(codes, scale, off=0, lds=None):
    """Device copies whose scales' rows are `lds` bytes apart (default: close together), with NaN
    scales around and between them."""
    R, kb = scale.shape
    lds = kb if lds is None else lds
    buf = np.full(off + R * lds + 16, 255, dtype=np.uint8)
    np.lib.stride_tricks.as_strided(buf[off:], (R, kb), (lds, 1))[:] = scale
    return to_dev(codes), to_dev(buf)[off:].as_strided((R, kb), (lds, 1))


# Every form of the kernel for few rows (1, 4, 16, 32, 48, 64 rows; more than eight runs of 512),
# tiles above; K with whole and cut last runs, and less than one
@pytest.mark.parametrize("M", [1, 3, 4, 5, 16, 17, 33, 49, 64, 65, 200, 300])
def test_scales_of_any_layout(gpu, M):
    for N, K in ((50, 40), (70, 300), (130, 500), (300, 1064), (130, 2880), (40, 4700)):
        rng = np.random.default_rng(M * 100 + K)
        A, sa = mx.random_matrix(rng, M, K, 118, 126)
        B, sb = mx.random_matrix(rng, N, K, 118, 126)
        x = rng.standard_normal((M, K)).astype(np.float16)
        ref, tol = mx.product(mx.values(A, sa), mx.values(B, sb))
        ref16, tol16 = mx.product(x.astype(np.float64), mx.values(B, sb)[:, :K])
        for off, lds in ((0, None), (1, None), (7, sb.shape[1] + 3), (16, None)):
            what = f"{M}x{N}x{K} scales at {off}, stride {lds}"
            log(what)
            a, b = close(A, sa, off, lds and sa.shape[1] + 3), close(B, sb, off, lds)
            for cfg in (None, tg.MX_SKINNY) if M <= tg.MX_SKINNY_ROWS else (None,):
                mx.check(tg.mxfp4_gemm(*a, *b, cfg=cfg).cpu().numpy(), ref, tol, what)
                mx.check(tg.mxfp4_gemm(*padded(A, sa), *b, cfg=cfg).cpu().numpy(), ref, tol, what)
                mx.check(tg.mxfp4_gemm_f16(to_dev(x), *b, cfg=cfg).cpu().numpy(), ref16, tol16, what)


def test_a_cloned_weight_is_the_weight(gpu):
    """clone and contiguous of the package's own scales, the autograd forms, another stream, a graph."""
    gen = gpu.Generator(device="cuda").manual_seed(5)
    x, w = (gpu.randn(s, generator=gen, device="cuda").half() for s in ((300, 1064), (520, 1064)))
    q, s = tg.mxfp4_quant(w)
    c = s.contiguous().clone()
    assert s.stride(0) == 48 and c.stride(0) == 34
    want = tg.mxfp4_gemm_f16(x, q, s)
    assert gpu.equal(tg.mxfp4_gemm_f16(x, q, c), want)
    assert gpu.equal(tg.mxfp4_linear(x, q, c), tg.mxfp4_linear(x, q, s))
    xg = x.clone().requires_grad_()
    for scale in (s, c):
        y = tg.Mxfp4WeightFunction.apply(xg, q, scale)
        g, = gpu.autograd.grad(y, xg, want)
        first = g if scale is s else first
        assert gpu.equal(y, want) and gpu.equal(g, first)
    side = gpu.cuda.Stream()
    side.wait_stream(gpu.cuda.current_stream())
    out = tg.mxfp4_gemm_f16(x, q, c, stream=side)
    side.synchronize()
    assert gpu.equal(out, want)
    graph = gpu.cuda.CUDAGraph()
    static = gpu.zeros_like(x)
    with gpu.cuda.graph(graph, stream=side):
        y = tg.mxfp4_gemm_f16(static, q, c)
        z = tg.mxfp4_linear(static, q, c)
    for i in range(3):
        static.copy_(x * (i + 1))
        graph.replay()
        gpu.cuda.synchronize()
        assert gpu.equal(y, tg.mxfp4_gemm_f16(x * (i + 1), q, s)) and gpu.equal(z, tg.mxfp4_linear(x * (i + 1), q, s))
