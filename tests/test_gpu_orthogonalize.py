"""The Newton-Schulz orthogonalisation on the GPU against its definition in float64, and as the
last part of a linear layer's training step.

Tolerance, in Frobenius norms relative to the exact result. One step rounds hi(X) (relative
2^-11 at most, about 2^-12 rms), the off-diagonals of A and of the polynomial, and the result;
each is a sum of independent roundings. The step's derivative at a singular value s is a + 3 b
s^2 + 5 c s^4, at most a = 3.4445 in magnitude over [0, 1.2], with a s the dominant part for the
small values it amplifies most, where hi(X)'s rounding enters only through offdiag(P) (small
there). Three roundings of 2^-12 rms per step, grown by at most 3.4445 once more in the following
step before the map contracts (|p'| < 1 around s = 0.9), give 5 * 3 * 2^-12 * 3.4445 = 1.3e-2
at worst; independent signs give sqrt(15) * 2^-12 * 3.4445 = 3.3e-3, which is the bound used."""
import numpy as np
import pytest

import mx_reference as mx
from gpu_util import log, to_dev, torch_cuda

import tiled_dense_gemm_04_amd as tg

pytestmark = pytest.mark.gpu

A, B, C = 3.4445, -4.7750, 2.0315
BOUND = np.sqrt(15) * 2.0 ** -12 * 3.4445


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = torch_cuda()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tg.lib()
    return torch


def reference(g, steps=5, scale=1.0, coefficients=(A, B, C)):
    """numpy float64, one matrix."""
    a, b, c = coefficients
    x = g.astype(np.float64)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (np.sqrt((x * x).sum()) + 1e-7)
    for _ in range(steps):
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return scale * (x.T if tall else x)


def distance(got, ref):
    return np.linalg.norm(got.astype(np.float64) - ref) / max(np.linalg.norm(ref), 1e-30)


def gradient(rng, R, C):
    return (rng.standard_normal((R, 4)) @ rng.standard_normal((4, C)) * 1e-3 + rng.standard_normal((R, C)) * 3e-3)


SHAPES = [(1, 1), (1, 300), (300, 1), (7, 5), (64, 64), (65, 200), (200, 65), (128, 128), (130, 129), (256, 1000),
          (1000, 256), (520, 392), (1024, 1024)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_against_definition(gpu, shape):
    rng = np.random.default_rng(shape[0] * 31 + shape[1])
    g = gradient(rng, *shape)
    for dtype in (np.float16, np.float32):
        x = g.astype(dtype)
        for steps in (1, 5):
            got = tg.orthogonalize(to_dev(x), steps=steps).cpu().numpy()
            d = distance(got, reference(x, steps))
            log(f"{shape} {dtype.__name__} steps {steps}: {d:.2e}")
            assert d <= BOUND


def test_singular_values_and_random_matrices(gpu):
    rng = np.random.default_rng(5)
    for R, C in ((256, 256), (192, 700), (700, 192)):
        x = (rng.standard_normal((R, C)) * 0.02).astype(np.float32)
        got = tg.orthogonalize(to_dev(x)).cpu().numpy().astype(np.float64)
        assert distance(got, reference(x)) <= BOUND
        s = np.linalg.svd(got, compute_uv=False)
        assert s.max() < 1.25 and np.median(s) > 0.65


def test_stack_strides_and_in_place(gpu):
    rng = np.random.default_rng(8)
    for R, C in ((70, 100), (100, 70), (129, 260)):
        g = np.stack([gradient(rng, R, C) * 10.0 ** -i for i in range(3)]).astype(np.float16)
        want = [reference(m, 5, 0.25) for m in g]
        ld, st = C + 3, (R + 2) * (C + 3)
        buf = gpu.full((3 * st,), 7.0, dtype=gpu.float16, device="cuda")
        view = buf[1:].as_strided((3, R, C), (st, ld, 1))
        view.copy_(to_dev(g))
        out = gpu.full((3, R + 1, C + 5), 3.0, dtype=gpu.float16, device="cuda")
        tg.orthogonalize(view, scale=0.25, out=out[:, :R, :C])
        for i in range(3):
            assert distance(out[i, :R, :C].cpu().numpy(), want[i]) <= BOUND
        assert (out[:, R:] == 3.0).all() and (out[:, :, C:] == 3.0).all()
        one = tg.orthogonalize(to_dev(g[1]), scale=0.25)
        assert gpu.equal(one, out[1, :R, :C]), "a matrix alone and in a stack differ"
        tg.orthogonalize(view, scale=0.25, out=view)
        assert gpu.equal(view, out[:, :R, :C])
        assert (buf[0] == 7.0) and (buf[1:].as_strided((3, R, 3), (st, ld, 1), 1 + C) == 7.0).all()


def test_zero_and_nonfinite_and_huge(gpu):
    rng = np.random.default_rng(9)
    g = np.stack([np.zeros((80, 90)), gradient(rng, 80, 90), gradient(rng, 80, 90) * 1e25, gradient(rng, 80, 90) * 1e-20])
    g = g.astype(np.float32)
    bad = g[1].copy()
    bad[3, 4] = np.nan
    inf = g[1].copy()
    inf[79, 89] = np.inf
    got = tg.orthogonalize(to_dev(np.concatenate([g, bad[None], inf[None]]))).cpu().numpy()
    assert (got[0] == 0).all()
    for i in (1, 2):
        assert distance(got[i], reference(g[i])) <= BOUND
    # a norm far below the 1e-7 in the denominator: the result is the formula's, tiny
    assert np.abs(got[3].astype(np.float64) - reference(g[3])).max() <= 2.0 ** -24
    assert np.isnan(got[4]).all() and np.isnan(got[5]).all()


def test_coefficients_and_empty(gpu):
    rng = np.random.default_rng(10)
    x = gradient(rng, 96, 160).astype(np.float32)
    k = (1.5, -0.5, 0.0)
    got = tg.orthogonalize(to_dev(x), steps=8, coefficients=k).cpu().numpy()
    assert distance(got, reference(x, 8, 1.0, k)) <= BOUND
    for shape in ((0, 5, 6), (2, 0, 6), (2, 6, 0)):
        assert tg.orthogonalize(gpu.empty(shape, dtype=gpu.float16, device="cuda")).shape == shape
    with pytest.raises(tg.TgemmError):
        tg.orthogonalize(to_dev(x), steps=0)
    with pytest.raises(ValueError):
        tg.orthogonalize(to_dev(x), out=gpu.empty((96, 161), dtype=gpu.float16, device="cuda"))
    with pytest.raises(tg.TgemmError):
        tg.orthogonalize(to_dev(x), workspace=gpu.empty(4096, dtype=gpu.uint8, device="cuda"))


def test_deterministic_streams_and_stale_workspace(gpu):
    rng = np.random.default_rng(11)
    x = to_dev(gradient(rng, 300, 500).astype(np.float16))
    ref = tg.orthogonalize(x)
    ws = gpu.full((tg.orthogonalize_workspace_bytes(1, 300, 500),), 255, dtype=gpu.uint8, device="cuda")
    gpu.cuda.synchronize()
    assert gpu.equal(tg.orthogonalize(x, workspace=ws), ref), "stale workspace contents leak in"
    side = gpu.cuda.Stream()
    for s in (side, side.cuda_stream):
        out = tg.orthogonalize(x, stream=s)
        side.synchronize()
        assert gpu.equal(out, ref)


def test_graph_replays(gpu):
    rng = np.random.default_rng(12)
    x = gpu.zeros((130, 200), dtype=gpu.float16, device="cuda")
    tg.orthogonalize(x)
    side = gpu.cuda.Stream()
    side.wait_stream(gpu.cuda.current_stream())
    g = gpu.cuda.CUDAGraph()
    with gpu.cuda.graph(g, stream=side):
        y = tg.orthogonalize(x)
    for i in range(4):
        x.copy_(to_dev(gradient(rng, 130, 200).astype(np.float16)))
        g.replay()
        gpu.cuda.synchronize()
        assert gpu.equal(y, tg.orthogonalize(x)), f"replay {i}"


def test_training_step(gpu):
    """A linear layer's whole step on the library: MXFP4 forward and gradients, momentum, and
    the weight moved along the orthogonalised momentum; then the new weight quantised and served
    to single tokens."""
    M, N, K = 200, 160, 260
    rng = np.random.default_rng(20)
    x = (rng.standard_normal((M, K))).astype(np.float16)
    w = (rng.standard_normal((N, K)) / 16).astype(np.float16)
    dy = (rng.standard_normal((M, N)) * 0.01).astype(np.float16)
    xd, wd = to_dev(x).requires_grad_(), to_dev(w).requires_grad_()
    y = tg.Mxfp4LinearFunction.apply(xd, wd)
    gx, gw = gpu.autograd.grad(y, (xd, wd), to_dev(dy))

    def q(v):
        v = np.ascontiguousarray(v)
        return mx.values(*mx.quant(v))[:, :v.shape[1]]

    for got, a, b in ((y.detach(), q(x), q(w)), (gx, q(dy), q(w.T)), (gw, q(dy.T), q(x.T))):
        mx.check(got.cpu().numpy(), *mx.product(a, b))
    momentum = gpu.zeros((N, K), dtype=gpu.float32, device="cuda").mul_(0.95).add_(gw.float())
    update = tg.orthogonalize(momentum, scale=0.02)
    assert distance(update.cpu().numpy(), reference(momentum.cpu().numpy(), 5, 0.02)) <= BOUND
    with gpu.no_grad():
        wd -= update
    codes, scale = tg.mxfp4_quant(wd.detach())
    wq = mx.values(*mx.quant(wd.detach().cpu().numpy()))[:, :K]
    for tokens in (1, 5):
        t = rng.standard_normal((tokens, K)).astype(np.float16)
        out = tg.mxfp4_gemm_f16(to_dev(t), codes, scale)
        mx.check(out.cpu().numpy(), *mx.product(t.astype(np.float64), mx.to_half(wq).astype(np.float64)))
        assert gpu.equal(tg.mxfp4_linear(to_dev(t), codes, scale),
                         tg.mxfp4_gemm(*tg.mxfp4_quant(to_dev(t)), codes, scale))


def test_poisoned_copies(gpu):
    """On the build that fills every LDS copy's destination with NaN bytes first, results stay
    the same bit for bit (wide and tall, tiles of 128 and of 256)."""
    rng = np.random.default_rng(44)
    for shape in ((3, 200, 333), (2, 333, 200), (40, 500, 520), (40, 520, 500)):
        g = to_dev(rng.standard_normal(shape).astype(np.float32))
        log(f"poisoned copies {shape}")
        assert gpu.equal(tg.orthogonalize(g, library=tg.debugfill_lib()), tg.orthogonalize(g))
