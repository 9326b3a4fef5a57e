"""The norm at the ends of its ranges: rows whose squares approach the ends of float32."""
import numpy as np
import pytest

import norm_reference as ref
from gpu_util import to_dev, torch_cuda

import tiled_dense_gemm_04_amd as tg

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = torch_cuda()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tg.lib()
    return torch


def rows_of_size(R, K, rms, seed=0):
    """float32 rows of normal values with this root mean square."""
    v = np.random.default_rng(seed).standard_normal((R, K))
    return (v * (rms / np.sqrt((v * v).mean(1, keepdims=True)))).astype(np.float32)


@pytest.mark.parametrize("K", [1, 100, 1000, 4096, 16384])
def test_rows_on_either_side_of_the_largest_sum_of_squares(gpu, K):
    """The documented end: a sum of squares up to float32's largest is as exact as any, one above gives zeros."""
    end = np.sqrt(float(np.finfo(np.float32).max) / K)
    x, w = np.zeros((3, K), dtype=np.float16), (1 + 0.2 * np.random.default_rng(1).standard_normal(K)).astype(np.float16)
    # the sum's error is below 2^-18 of it: 0.1 per cent to either side is clear of the end
    r = rows_of_size(3, K, 0.999 * end)
    y, h = tg.rmsnorm(to_dev(x), to_dev(w), to_dev(r), eps=EPS)
    assert np.array_equal(h.cpu().numpy(), r)
    want, _ = ref.norm(r, w, EPS)
    assert (np.abs(y.cpu().numpy() - want) <= ref.y_bound(want)).all()
    leaves = [to_dev(t).requires_grad_() for t in (x, w, r)]
    dy = (0.1 * np.random.default_rng(2).standard_normal((3, K))).astype(np.float16)
    y, h = tg.RmsNormFunction.apply(*leaves, EPS)
    _, dw, dr = gpu.autograd.grad((y, h), leaves, (to_dev(dy), to_dev(np.zeros((3, K), dtype=np.float32))))
    dx, bound, dw64, size = ref.gradient(dy, r, w, EPS)
    assert (np.abs(dr.cpu().numpy() - dx) <= bound + np.abs(dx) * 2.0 ** -18 + 2.0 ** -126).all()
    # three rows' products and sums: below 16 roundings of 2^-24
    assert (np.abs(dw.cpu().numpy() - dw64) <= size * 2.0 ** -18 + np.abs(dw64) * ref.HALF16 + ref.TINY16).all()
    r = rows_of_size(3, K, 1.001 * end)
    y, h = tg.rmsnorm(to_dev(x), to_dev(w), to_dev(r), eps=EPS)
    q, s, _ = tg.rmsnorm_fp8_block(to_dev(x), to_dev(w), to_dev(r), eps=EPS)
    assert np.array_equal(h.cpu().numpy(), r)
    assert (y == 0).all() and (q.cpu().numpy() & 127 == 0).all() and (s == 1).all()


def test_rows_without_eps(gpu):
    """eps = 0: rows of zeros are NaN, small ones exact as long as their squares are normal numbers, and
    infinite once all of those are 0."""
    K = 512
    x, w = np.zeros((1, K), dtype=np.float16), np.ones(K, dtype=np.float16)
    assert gpu.isnan(tg.rmsnorm(to_dev(x), to_dev(w), eps=0.0)).all()
    r = rows_of_size(1, K, 1e-18)
    r[np.abs(r) < 2e-19] = 2e-19
    want, _ = ref.norm(r, w, 0.0)
    assert (np.abs(tg.rmsnorm(to_dev(x), to_dev(w), to_dev(r), eps=0.0)[0].cpu().numpy() - want) <= ref.y_bound(want)).all()
    r = np.full((1, K), 2.5e-23, dtype=np.float32)
    assert gpu.isinf(tg.rmsnorm(to_dev(x), to_dev(w), to_dev(r), eps=0.0)[0]).all()
