"""MXFP4 products whose float32 sums are exact, so that every kernel's result is the exact one rounded
once, bit for bit: a single code, scale or row that is dropped, read twice or taken from a wrong
place along a long K shows."""
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
    s = np.full((len(scale), -(-scale.shape[1] // 16) * 16), 255, dtype=np.uint8)
    s[:, :scale.shape[1]] = scale
    return to_dev(codes), to_dev(s)[:, :scale.shape[1]]


def exact(a, b, unit):
    """float16 of a b^T; every partial sum is a multiple of `unit` below 2^24 of it: a float32."""
    assert (np.abs(a) @ np.abs(b).T).max() < unit * 2.0 ** 24
    c = (a @ b.T).astype(np.float16)
    assert np.isfinite(c).all()
    return c


# Cut last k-tiles, scale groups and runs, and many turns of every ring
SIZES = [(1, 40, 8200), (5, 33, 8192), (37, 70, 4128), (64, 130, 6000), (200, 264, 4128), (130, 260, 8200), (520, 300, 4700),
         (1000, 513, 2080)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_exact_sums(gpu, M, N, K):
    rng = np.random.default_rng(M + K)
    # codes in quarters of 2^-3 .. 2^-1 (scales 124 .. 126): products are multiples of 2^-8
    A, sa = mx.random_matrix(rng, M, K, 124, 126)
    B, sb = mx.random_matrix(rng, N, K, 124, 126)
    want = exact(mx.values(A, sa), mx.values(B, sb), 2.0 ** -8)
    for cfg in (None, tg.MX_GENERIC, tg.MX_SKINNY, tg.MX_64, tg.MX_128, tg.MX_256):
        if cfg == tg.MX_SKINNY and M > tg.MX_SKINNY_ROWS:
            continue
        log(f"{M}x{N}x{K} kernel {cfg}")
        c = tg.mxfp4_gemm(*padded(A, sa), *padded(B, sb), cfg=cfg).cpu().numpy()
        assert np.array_equal(c, want), f"kernel {cfg}: {(c != want).sum()} values differ"


@pytest.mark.parametrize("M,N,K", SIZES)
def test_exact_sums_f16(gpu, M, N, K):
    rng = np.random.default_rng(M + K + 1)
    a = (rng.integers(-32, 33, (M, K)) / 8).astype(np.float16)   # multiples of 2^-3
    B, sb = mx.random_matrix(rng, N, K, 124, 126)                # multiples of 2^-4
    want = exact(a.astype(np.float64), mx.values(B, sb)[:, :K], 2.0 ** -7)
    for cfg in (None, tg.MX_GENERIC, tg.MX_SKINNY, tg.MX_128, tg.MX_256):
        if (cfg == tg.MX_SKINNY and M > tg.MX_SKINNY_ROWS) or (cfg in (tg.MX_128, tg.MX_256) and K % 8):
            continue
        log(f"{M}x{N}x{K} kernel {cfg}")
        c = tg.mxfp4_gemm_f16(to_dev(a), *padded(B, sb), cfg=cfg).cpu().numpy()
        assert np.array_equal(c, want), f"kernel {cfg}: {(c != want).sum()} values differ"


@pytest.mark.parametrize("M,N,K", [(300, 200, 4100), (4096, 96, 264), (65, 8192, 130)])
def test_exact_gradients(gpu, M, N, K):
    """The three products of a training step, inputs on the grid with a long inner dimension each."""
    rng = np.random.default_rng(N)
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, -0.5, -1, -1.5, -2, -3, -4])
    x, w, dy = (rng.choice(grid, s) for s in ((M, K), (N, K), (M, N)))
    # (a block whose largest value is below 4 has a finer grid: inputs stay themselves)
    xd, wd = (to_dev(v.astype(np.float16)).requires_grad_() for v in (x, w))
    y = tg.Mxfp4LinearFunction.apply(xd, wd)
    gx, gw = gpu.autograd.grad(y, (xd, wd), to_dev(dy.astype(np.float16)))
    for name, got, a, b in (("y", y.detach(), x, w), ("dx", gx, dy, w.T), ("dw", gw, dy.T, x.T)):
        assert np.array_equal(got.cpu().numpy(), exact(a, b, 0.25)), name
