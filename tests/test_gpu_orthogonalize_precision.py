"""What the orthogonalisation loses, against float64 with the bound of ns_reference: matrices with
few and many strong directions, four to ten steps, wide and tall, and every tile size of its three
products."""
import numpy as np
import pytest

import ns_reference as ns
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


def check(got, g, steps, what):
    """got: the result for g (wide or tall), float16 numpy."""
    ref = ns.iterates(g, steps)[-1]
    got = got.astype(np.float64)
    err = np.linalg.norm((got.T if got.shape != ref.shape or g.shape[0] > g.shape[1] else got) - ref)
    bound = ns.bound(g, ref, steps)
    log(f"{what}: error {err / np.linalg.norm(ref):.2e}, bound {bound / np.linalg.norm(ref):.2e}")
    assert err <= bound, what


SHAPES = [(1, 1), (1, 300), (7, 5), (64, 64), (64, 500), (65, 200), (130, 129), (256, 256), (256, 1000), (512, 512)]


@pytest.mark.parametrize("name", ns.INPUTS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_inputs_and_steps(gpu, shape, name):
    g = ns.INPUTS[name](np.random.default_rng(shape[0] * 7 + shape[1]), *shape)
    for dtype, x in ((np.float32, g), (np.float16, g.T)):
        x = np.ascontiguousarray(x.astype(dtype))
        for steps in (4, 5, 6, 10):
            got = tg.orthogonalize(to_dev(x), steps=steps).cpu().numpy()
            check(got, x, steps, f"{name} {x.shape} {dtype.__name__} {steps} steps")


def test_large(gpu):
    for shape in ((1024, 1024), (2048, 700)):
        x = ns.directions(np.random.default_rng(3), *shape).astype(np.float32)
        check(tg.orthogonalize(to_dev(x)).cpu().numpy(), x, 5, f"{shape}")


# A product takes tiles of 256 x 256 where its batch has 128 or more of them (the symmetric ones: on
# and above the diagonal), else of 128 x 128: here all three on 256, one, three and six tiles of A
# each; then Apply alone on 256.
STACKS = [(128, 256, 320), (43, 300, 520), (22, 640, 700), (40, 200, 900)]


@pytest.mark.parametrize("shape", STACKS, ids=str)
@pytest.mark.parametrize("tall", [False, True], ids=["wide", "tall"])
def test_stacks_on_large_tiles(gpu, shape, tall):
    batch, m, n = shape
    rng = np.random.default_rng(m + n)
    names = list(ns.INPUTS)
    g = np.stack([ns.INPUTS[names[i % len(names)]](rng, m, n) for i in range(batch)]).astype(np.float32)
    g = np.ascontiguousarray(g.transpose(0, 2, 1)) if tall else g
    got = tg.orthogonalize(to_dev(g)).cpu().numpy()
    for i in sorted({0, 1, 2, 3, 4, batch // 2, batch - 2, batch - 1}):
        check(got[i], g[i], 5, f"{g.shape} matrix {i}")
    for i in range(batch):  # the others against the small tiles' results, which differ in summation order only
        one = tg.orthogonalize(to_dev(g[i])).cpu().numpy().astype(np.float64)
        assert np.linalg.norm(got[i] - one) <= 1e-3 * np.linalg.norm(one), f"matrix {i}"


@pytest.mark.parametrize("shape", [(43, 300, 520), (43, 520, 300)], ids=str)
def test_poisoned_copies_on_large_tiles(gpu, shape):
    """On the build that fills every LDS copy's destination with NaN bytes first, the symmetric
    products on 256 x 256 tiles stay the same bit for bit; a NaN stays in its own matrix."""
    g = to_dev(np.random.default_rng(9).standard_normal(shape).astype(np.float32))
    want = tg.orthogonalize(g)
    assert gpu.equal(tg.orthogonalize(g, library=tg.debugfill_lib()), want)
    g[7, 150, 200] = float("nan")
    got = tg.orthogonalize(g)
    assert gpu.isnan(got[7]).all()
    for i in (0, 6, 8, 42):
        assert gpu.equal(got[i], want[i])
