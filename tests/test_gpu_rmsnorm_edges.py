"""The norm at the ends of its ranges: rows whose squares approach the ends of float32, and gradients
of so many rows that every workgroup goes over several in turn."""
import numpy as np
import pytest

import norm_reference as ref
from gpu_util import to_dev, torch_cuda
from test_gpu_rmsnorm import check_codes, check_y

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
    leaves = [to_dev(t).requires_grad_() for t in (x, w, r)]
    dx, dw, dr = gpu.autograd.grad(tg.RmsNormFunction.apply(*leaves, EPS), leaves, (to_dev(dy), to_dev(dy.astype(np.float32))))
    assert np.array_equal(dx.cpu().numpy(), dy) and (dw == 0).all() and np.array_equal(dr.cpu().numpy(), dy.astype(np.float32))


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


# (rows, columns, turns of the longest workgroup, rows it holds at once): past the most workgroups that the
# backward kernel has (1024 of 256 threads, 512 of 512, 256 of 1024), with a last turn that is not full,
# for every number of threads a row.
MANY_ROWS = [(40000, 128, 3, 16), (16391, 200, 3, 8), (12290, 520, 4, 4), (9001, 777, 3, 4), (5125, 1032, 6, 1), (3077, 1100, 4, 1),
             (3077, 2100, 4, 1), (1539, 4104, 4, 1), (769, 8200, 4, 1), (2049, 16383, 9, 1)]


@pytest.mark.parametrize("residual", [None, np.float16, np.float32], ids=lambda r: "none" if r is None else r.__name__)
@pytest.mark.parametrize("R, K, turns, at_once", MANY_ROWS, ids=str)
def test_gradient_of_many_rows(gpu, R, K, turns, at_once, residual):
    groups = tg.lib().rmsnorm_f16_backward_workspace_bytes(R, K) // (4 * K)
    assert -(-R // (groups * at_once)) == turns and groups < -(-R // (2 * at_once))
    rng = np.random.default_rng(R + K)
    x, dy = (rng.standard_normal((R, K), dtype=np.float32).astype(np.float16) for _ in range(2))
    r, dh = (None, None) if residual is None else (rng.standard_normal((R, K), dtype=np.float32).astype(residual) for _ in range(2))
    w = (1 + 0.2 * rng.standard_normal(K)).astype(np.float32 if K % 2 else np.float16)
    leaves = [to_dev(t).requires_grad_() for t in (x, w)] + ([] if r is None else [to_dev(r).requires_grad_()])

    def grads():
        if r is None:
            return gpu.autograd.grad(tg.RmsNormFunction.apply(*leaves, None, EPS), leaves, to_dev(dy))
        return gpu.autograd.grad(tg.RmsNormFunction.apply(*leaves, EPS), leaves, (to_dev(dy), to_dev(dh)))

    got = grads()
    h = ref.stored(x, r)
    dx, bound, dw, size = ref.gradient(dy, h, w, EPS, dh)
    assert (np.abs(got[0].cpu().numpy() - dx) <= bound + np.abs(dx) * (ref.HALF16 + 2.0 ** -18) + ref.TINY16).all()
    if r is not None:
        step, tiny = (ref.HALF16, ref.TINY16) if residual == np.float16 else (2.0 ** -24, 0.0)
        assert (np.abs(got[2].cpu().numpy() - dx) <= bound + np.abs(dx) * (step + 2.0 ** -18) + tiny).all()
    # a thread adds up to 9 rows, up to 16 of its workgroup's threads are joined, then up to 1024 / 16 partial
    # sums a wave and 16 waves: 105 roundings of 2^-24; the product, xhat and rstd (28) 30 more: below 2^-16
    tol = size * 2.0 ** -16 + (0.0 if w.dtype == np.float32 else 1.0) * (np.abs(dw) * ref.HALF16 + ref.TINY16)
    assert (np.abs(got[1].cpu().numpy() - dw) <= tol).all()
    # which sees a row of the last turn left out
    xhat = h[-1].astype(np.float64) / np.sqrt((h[-1].astype(np.float64) ** 2).mean() + EPS)
    assert (np.abs(dy[-1] * xhat) > size * 2.0 ** -16 + (0.0 if w.dtype == np.float32 else 1.0) * np.abs(dw) * ref.HALF16).any()
    assert all(gpu.equal(a, b) for a, b in zip(got, grads()))  # sums in a fixed order


@pytest.mark.parametrize("residual", [np.float16, np.float32], ids=lambda r: r.__name__)
@pytest.mark.parametrize("rows", [2047, 2048])
def test_rows_of_six_waves(gpu, rows, residual):
    """Both sides of the choice of six waves a row: every row end, strided and in place, y and codes."""
    for K in (2559, *range(2560, 2569), 3000, 3064, 3071, 3073):
        rng = np.random.default_rng(K)
        x = rng.standard_normal((rows, K), dtype=np.float32).astype(np.float16)
        r = (3 * rng.standard_normal((rows, K), dtype=np.float32)).astype(residual)
        w = (1 + 0.2 * rng.standard_normal(K)).astype(np.float32 if K % 2 else np.float16)
        h = ref.stored(x, r)
        xd, wd = to_dev(x), to_dev(w)
        wide = gpu.full((rows, K + 5), 7.0, dtype=to_dev(r).dtype, device="cuda")
        wide[:, 3:K + 3] = to_dev(r)
        out = gpu.full((rows, K + 3), 5.0, dtype=gpu.float16, device="cuda")
        q, s, coded = tg.rmsnorm_fp8_block(xd, wd, wide[:, 3:K + 3], eps=EPS)
        tg.rmsnorm(xd, wd, wide[:, 3:K + 3], eps=EPS, out=out[:, 1:K + 1], residual_out=wide[:, 3:K + 3])
        check_y(out[:, 1:K + 1], h, w)
        check_codes(q, s, h, w)
        assert np.array_equal(wide[:, 3:K + 3].cpu().numpy(), h) and np.array_equal(coded.cpu().numpy(), h), K
        assert (wide[:, :3] == 7).all() and (wide[:, K + 3:] == 7).all() and (out[:, 0] == 5).all() and (out[:, K + 1:] == 5).all()
