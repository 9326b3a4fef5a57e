"""The root-mean-square norm on the GPU against float64 (norm_reference): every row shape of the
kernels, residual and weight types, ragged sizes, strides and alignments, in-place updates, special
values, the E4M3 output and the product it feeds, the gradient against its formula and against
differences, streams, graphs and saved-tensor hooks."""
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


def case(R, K, residual, w32=False, seed=0):
    rng = np.random.default_rng(1000 * R + K + seed)
    gain = np.where(rng.random(K) < 0.02, 12.0, 1.0)
    x = (rng.standard_normal((R, K)) * gain).astype(np.float16)
    r = None if residual is None else (3 * rng.standard_normal((R, K)) * gain).astype(residual)
    w = (1 + 0.2 * rng.standard_normal(K)).astype(np.float32 if w32 else np.float16)
    return x, r, w


def check_y(y, h, w):
    want, _ = ref.norm(h, w, EPS)
    got = y.cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= ref.y_bound(want)).all()


def check_codes(q, s, h, w):
    want, _ = ref.norm(h, w, EPS)
    scale, lo, hi = ref.codes_range(want)
    assert (np.abs(s.cpu().numpy() - scale) <= scale * 2.0 ** -18).all()
    v = ref.e4m3_value(q.cpu().numpy())
    assert ((lo <= v) & (v <= hi)).all()


# Every row shape of the kernels (16 to 1024 threads, one and two chunks), their edges, ragged K.
SHAPES = [(1, 1), (3, 7), (1, 8), (5, 127), (37, 128), (6, 129), (35, 200), (9, 256), (5, 257), (4, 512), (7, 513), (1, 1000), (5, 1024), (3, 1025),
          (300, 130), (2, 2048), (3, 2049), (5, 3000), (1, 4096), (2, 4097), (2, 5000), (3, 8192), (2, 8193), (1, 16383),
          (2, 16384)]


@pytest.mark.parametrize("residual", [None, np.float16, np.float32], ids=lambda r: "none" if r is None else r.__name__)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm(gpu, shape, residual):
    x, r, w = case(*shape, residual, w32=shape[1] % 2 == 1)
    xd, wd, rd = to_dev(x), to_dev(w), None if r is None else to_dev(r)
    h = ref.stored(x, r)
    got, coded = tg.rmsnorm(xd, wd, rd, eps=EPS), tg.rmsnorm_fp8_block(xd, wd, rd, eps=EPS)
    check_y(got if r is None else got[0], h, w)
    check_codes(coded[0], coded[1], h, w)
    if r is not None:
        assert np.array_equal(got[1].cpu().numpy(), h) and np.array_equal(coded[2].cpu().numpy(), h)
        assert np.array_equal(rd.cpu().numpy(), r)


@pytest.mark.parametrize("residual", [None, np.float16, np.float32], ids=lambda r: "none" if r is None else r.__name__)
def test_every_row_end(gpu, residual):
    """Rows that end in every place of a chunk of eight, up to one chunk, past it, and in the shapes of 4 and 6
    waves a row; forward and backward."""
    for K in [*range(2, 18), 2559, *range(2561, 2568), 3071, 3073]:
        x, r, w = case(3, K, residual, w32=K % 2 == 1)
        xd, wd, rd = to_dev(x), to_dev(w), None if r is None else to_dev(r)
        h = ref.stored(x, r)
        got, coded = tg.rmsnorm(xd, wd, rd, eps=EPS), tg.rmsnorm_fp8_block(xd, wd, rd, eps=EPS)
        check_y(got if r is None else got[0], h, w)
        check_codes(coded[0], coded[1], h, w)
        if r is not None:
            assert np.array_equal(got[1].cpu().numpy(), h), K
        test_gradient(gpu, (3, K), residual)


def test_strides_alignment_and_untouched_memory(gpu):
    for K in (1000, 129, 4100):
        x, r, w = case(6, K, np.float32)
        buf = gpu.full((6, K + 3), 7.0, dtype=gpu.float16, device="cuda")
        buf[:, 1:K + 1] = to_dev(x)
        rb = gpu.full((6, K + 5), 7.0, dtype=gpu.float32, device="cuda")
        rb[:, 3:K + 3] = to_dev(r)
        wb = gpu.ones(K + 1, dtype=gpu.float16, device="cuda")
        wb[1:] = to_dev(w)
        y = gpu.full((6, K + 7), 5.0, dtype=gpu.float16, device="cuda")
        q = gpu.full((6, K + 9), 77, dtype=gpu.uint8, device="cuda")
        h = ref.stored(x, r)
        tg.rmsnorm(buf[:, 1:K + 1], wb[1:], rb[:, 3:K + 3], eps=EPS, out=y[:, 3:K + 3], residual_out=rb[:, 3:K + 3])
        check_y(y[:, 3:K + 3], h, w)
        assert np.array_equal(rb[:, 3:K + 3].cpu().numpy(), h)  # updated in place
        assert (rb[:, :3] == 7).all() and (rb[:, K + 3:] == 7).all() and (y[:, :3] == 5).all() and (y[:, K + 3:] == 5).all()
        _, s = tg.rmsnorm_fp8_block(rb[:, 3:K + 3].half().contiguous(), wb[1:], eps=EPS, q=q[:, 1:K + 1])
        check_codes(q[:, 1:K + 1], s, h.astype(np.float16), w)
        assert (q[:, 0] == 77).all() and (q[:, K + 1:] == 77).all()
        xin = buf[:, 1:K + 1]
        tg.rmsnorm(xin, wb[1:], eps=EPS, out=xin)  # in place of x
        check_y(xin, x, w)


def test_special_values(gpu):
    K = 300
    x, r, w = case(8, K, np.float16)
    x[0] = 0
    r[0] = 0                                            # a row of zeros: zeros, with eps > 0
    x[1, 5], x[2, 200], x[3, 299] = np.inf, np.nan, -np.inf
    x[4], r[4] = 65504, -65504                          # the sum is exact where both parts are large
    r[5] = 6e-8                                         # subnormal sums
    x[5] = 0
    q, s, h = tg.rmsnorm_fp8_block(to_dev(x), to_dev(w), to_dev(r), eps=EPS)
    y, h2 = tg.rmsnorm(to_dev(x), to_dev(w), to_dev(r), eps=EPS)
    want_h = ref.stored(x, r)
    assert np.array_equal(h.cpu().numpy(), want_h, equal_nan=True) and np.array_equal(h2.cpu().numpy(), want_h, equal_nan=True)
    y, q, s = y.cpu().numpy(), q.cpu().numpy(), s.cpu().numpy()
    assert (y[0] == 0).all() and (q[0] == 0).all() and (s[0] == 1).all()
    # an infinity: rstd 0, so NaN where it stands and zeros elsewhere; its block is marked
    assert np.isnan(y[1, 5]) and (np.delete(y[1], 5) == 0).all() and np.isnan(s[1, 0]) and (q[1] == 0).all()
    assert np.isnan(y[2]).all() and np.isnan(s[2]).all() and (q[2] == 0).all()
    assert np.isnan(s[3, 2]) and (s[3, :2] == 1).all()
    good = [4, 5, 6, 7]
    want, _ = ref.norm(want_h[good], w, EPS)
    assert (np.abs(y[good] - want) <= ref.y_bound(want)).all()
    # float32 residuals below binary16's range; a block below 2^-100 counts as zeros
    r = np.zeros((2, 256), dtype=np.float32)
    r[0, :128], r[0, 128:] = 1e-30, 1e-38
    r[1] = 1e-20
    zero, one = np.zeros((2, 256), dtype=np.float16), np.ones(256, dtype=np.float16)
    q, s, h = tg.rmsnorm_fp8_block(to_dev(zero), to_dev(one), to_dev(r), eps=EPS)
    assert np.array_equal(h.cpu().numpy(), r)
    assert s.cpu().numpy()[0, 1] == 1 and (q.cpu().numpy()[0, 128:] == 0).all()
    check_codes(q[1:], s[1:], r[1:], one)


def test_codes_of_equal_values_and_the_grid(gpu):
    """Rows of one magnitude (every code is 448 or -448) and of a whole grid of ratios with a weight of
    ones, where many quotients are ties: each code is one of the two neighbours."""
    x = np.ones((3, 256), dtype=np.float16)
    x[1, ::2] = -1
    x[2, :128] = (np.arange(128) + 1) / 128 * 1.75
    x[2, 128:] = np.arange(128) * 2.0 ** -20
    one = np.ones(256, dtype=np.float32)
    q, s = tg.rmsnorm_fp8_block(to_dev(x), to_dev(one), eps=EPS)
    check_codes(q, s, x, one)
    assert (np.abs(ref.e4m3_value(q.cpu().numpy()[:2])) == 448).all()


def test_feeds_the_fp8_product(gpu):
    """rmsnorm_fp8_block into gemm_fp8_block: the product of the codes and scales it wrote."""
    import oracle
    M, N, K = 70, 200, 1040
    x, r, w = case(M, K, np.float16)
    rng = np.random.default_rng(5)
    wq, sw = tg.quant_fp8_block(to_dev((rng.standard_normal((N, K)) / 32).astype(np.float16)), 128)
    q, s, _ = tg.rmsnorm_fp8_block(to_dev(x), to_dev(w), to_dev(r), eps=EPS)
    c = tg.gemm_fp8_block(q, s, wq, sw)
    Q, S, W, SW = (t.cpu().numpy() for t in (q, s, wq, sw))
    rep = oracle.compare_fp8(c.cpu().numpy().view(np.uint16), oracle.gemm_fp8(Q, S, W, SW, False), oracle.fp8_bound(Q, S, W, SW))
    assert rep["fails"] == 0, rep


GRAD_SHAPES = [(1, 1), (300, 64), (1, 130), (41, 256), (5, 257), (5, 512), (6, 513), (2100, 1000), (3, 1025), (700, 2048), (5, 3000), (600, 4096), (3, 4097),
               (530, 8192), (2, 8193), (3, 16384)]


def check_grads(x, r, w, dy, dh, grads):
    h = ref.stored(x, r)
    dx, bound, dw, size = ref.gradient(dy, h, w, EPS, dh)
    got = grads[0].cpu().numpy().astype(np.float64)
    assert (np.abs(got - dx) <= bound + np.abs(dx) * (ref.HALF16 + 2.0 ** -18) + ref.TINY16).all()
    got = grads[1].cpu().numpy().astype(np.float64)
    # a group's rows (two or three here), up to 16 of its threads' sums, at most 1024 / 16 partial sums and 16
    # waves add up: below 100 roundings of 2^-24, and one of the product and of xhat each
    half = 0.0 if w.dtype == np.float32 else 1.0
    assert (np.abs(got - dw) <= size * 2.0 ** -17 + half * (np.abs(dw) * ref.HALF16 + ref.TINY16) + 2.0 ** -126).all()
    if r is not None:
        got = grads[2].cpu().numpy().astype(np.float64)
        step, tiny = (ref.HALF16, ref.TINY16) if r.dtype == np.float16 else (2.0 ** -24, 0.0)
        assert (np.abs(got - dx) <= bound + np.abs(dx) * (step + 2.0 ** -18) + tiny).all()


@pytest.mark.parametrize("residual", [None, np.float16, np.float32], ids=lambda r: "none" if r is None else r.__name__)
@pytest.mark.parametrize("shape", GRAD_SHAPES, ids=str)
def test_gradient(gpu, shape, residual):
    x, r, w = case(*shape, residual, w32=shape[1] % 4 == 0, seed=3)
    rng = np.random.default_rng(17)
    dy = (0.1 * rng.standard_normal(shape)).astype(np.float16)
    dh = None if r is None else (0.1 * rng.standard_normal(shape)).astype(residual)
    leaves = [to_dev(x).requires_grad_(), to_dev(w).requires_grad_()]
    if r is None:
        y = tg.RmsNormFunction.apply(*leaves, None, EPS)
        check_y(y.detach(), x, w)
        grads = gpu.autograd.grad(y, leaves, to_dev(dy))
    else:
        leaves.append(to_dev(r).requires_grad_())
        y, h = tg.RmsNormFunction.apply(*leaves, EPS)
        check_y(y.detach(), ref.stored(x, r), w)
        grads = gpu.autograd.grad((y, h), leaves, (to_dev(dy), to_dev(dh)))
    check_grads(x, r, w, dy, dh, grads)
    # the same again: sums in a fixed order
    if r is None:
        again = gpu.autograd.grad(tg.RmsNormFunction.apply(*leaves, None, EPS), leaves, to_dev(dy))
        assert all(gpu.equal(a, b) for a, b in zip(grads, again))


def test_gradient_against_differences(gpu):
    """Directional derivatives of the float64 definition by central differences."""
    R, K = 7, 200
    x, r, w = case(R, K, np.float32, w32=True, seed=9)
    x64 = ref.stored(x, r).astype(np.float64)
    rng = np.random.default_rng(2)
    dy, dh = (rng.standard_normal((R, K)).astype(t) for t in (np.float16, np.float32))
    leaves = [to_dev(x).requires_grad_(), to_dev(w).requires_grad_(), to_dev(r).requires_grad_()]
    y, h = tg.RmsNormFunction.apply(*leaves, EPS)
    gx, gw, gr = (g.cpu().numpy().astype(np.float64) for g in gpu.autograd.grad((y, h), leaves, (to_dev(dy), to_dev(dh))))
    assert (np.abs(gx - gr) <= np.abs(gr) * ref.HALF16 + ref.TINY16).all()

    def loss(h, w):
        return (ref.norm(h, w, EPS)[0] * dy.astype(np.float64)).sum() + (h * dh.astype(np.float64)).sum()

    t = 1e-5
    for _ in range(5):
        v, u = rng.standard_normal((R, K)), rng.standard_normal(K)
        num = (loss(x64 + t * v, w) - loss(x64 - t * v, w)) / (2 * t)
        # dr is float32 (relative 2^-18 of its magnitudes); the differences' own error is below 1e-6 of theirs
        assert abs(num - (gr * v).sum()) <= 1e-5 * np.abs(gr * v).sum() + 1e-5
        num = (loss(x64, w.astype(np.float64) + t * u) - loss(x64, w.astype(np.float64) - t * u)) / (2 * t)
        assert abs(num - (gw * u).sum()) <= 1e-5 * np.abs(gw * u).sum() + 1e-5


def test_partial_gradients(gpu):
    """Only some inputs want gradients, only one output is used, a broadcast gradient."""
    x, r, w = case(40, 520, np.float16)
    dy = np.full((40, 520), 0.25, dtype=np.float16)
    xd, wd, rd = to_dev(x), to_dev(w), to_dev(r)
    for need in ((True, False, False), (False, True, False), (False, False, True), (True, False, True)):
        leaves = [t.clone().requires_grad_(n) for t, n in zip((xd, wd, rd), need)]
        y, h = tg.RmsNormFunction.apply(*leaves, EPS)
        wanted = [t for t in leaves if t.requires_grad]
        got = gpu.autograd.grad(y, wanted, gpu.full((), 0.25, dtype=gpu.float16, device="cuda").expand(40, 520))
        full = [t.clone().requires_grad_() for t in (xd, wd, rd)]
        y, h = tg.RmsNormFunction.apply(*full, EPS)
        every = gpu.autograd.grad(y, full, to_dev(dy))
        check_grads(x, r, w, dy, None, every)
        assert all(gpu.equal(g, e) for g, e in zip(got, [e for e, n in zip(every, need) if n]))
    leaves = [t.clone().requires_grad_() for t in (xd, wd, rd)]
    _, h = tg.RmsNormFunction.apply(*leaves, EPS)  # only the updated residual is used
    dx, dw, dr = gpu.autograd.grad(h, leaves, to_dev(dy))
    assert (dx == 0.25).all() and (dw == 0).all() and (dr == 0.25).all()
    with pytest.raises(RuntimeError, match="second derivative"):
        y, _ = tg.RmsNormFunction.apply(*leaves, EPS)
        gpu.autograd.grad(y.float().sum(), leaves, create_graph=True)


def test_empty(gpu):
    x, w = gpu.empty((0, 64), dtype=gpu.float16, device="cuda"), gpu.ones(64, dtype=gpu.float16, device="cuda")
    assert tg.rmsnorm(x, w).shape == (0, 64)
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    dx, dw = gpu.autograd.grad(tg.RmsNormFunction.apply(xg, wg, None, EPS), (xg, wg), x)
    assert dx.shape == (0, 64) and (dw == 0).all()
    q, s = tg.rmsnorm_fp8_block(gpu.empty((5, 0), dtype=gpu.float16, device="cuda"), w[:0])
    assert q.shape == (5, 0) and s.shape == (5, 0)


def test_streams_and_graphs(gpu):
    """On another stream than the current one, and captured (a training step with leaves of its own):
    replays on new inputs give the eager results bit for bit."""
    x, r, w = case(300, 1000, np.float16)
    dy = to_dev((0.1 * np.random.default_rng(1).standard_normal((300, 1000))).astype(np.float16))
    inputs = [to_dev(x), to_dev(w), to_dev(r)]
    want = tg.rmsnorm(inputs[0], inputs[1], inputs[2])
    side = gpu.cuda.Stream()
    side.wait_stream(gpu.cuda.current_stream())
    got = tg.rmsnorm(inputs[0], inputs[1], inputs[2], stream=side)
    coded = tg.rmsnorm_fp8_block(inputs[0], inputs[1], inputs[2], stream=side.cuda_stream)
    side.synchronize()
    assert all(gpu.equal(a, b) for a, b in zip(want, got)) and gpu.equal(coded[2], want[1])

    def step(leaves):
        y, h = tg.RmsNormFunction.apply(*leaves, EPS)
        return (y, h, *gpu.autograd.grad((y, h), leaves, (dy, dy)))

    def eager(seed):
        x, r, w = case(300, 1000, np.float16, seed=seed)
        vals = [to_dev(x), to_dev(w), to_dev(r)]
        return vals, [t.detach().clone() for t in step([t.clone().requires_grad_() for t in vals])]

    static = [t.clone().requires_grad_() for t in inputs]
    with gpu.cuda.stream(side):
        step([t.clone().requires_grad_() for t in inputs])
    side.synchronize()
    graph = gpu.cuda.CUDAGraph()
    with gpu.cuda.graph(graph, stream=side):
        out = [t.detach() for t in step(static)]
    for seed in range(4):
        vals, expected = eager(seed)
        with gpu.no_grad():
            for s, v in zip(static, vals):
                s.copy_(v)
        graph.replay()
        gpu.cuda.synchronize()
        assert all(gpu.equal(a, b) for a, b in zip(out, expected)), seed


def test_saved_tensor_hooks(gpu):
    """Offloading hooks give the same gradients; a hook that returns another tensor is refused."""
    x, r, w = case(64, 520, np.float32)
    dy = to_dev(np.full((64, 520), 0.5, dtype=np.float16))

    def grads(pack, unpack):
        leaves = [to_dev(t).requires_grad_() for t in (x, w, r)]
        with gpu.autograd.graph.saved_tensors_hooks(pack, unpack):
            y, h = tg.RmsNormFunction.apply(*leaves, EPS)
        return gpu.autograd.grad(y, leaves, dy)

    plain = grads(lambda t: t, lambda t: t)
    moved = grads(lambda t: t.cpu(), lambda t: t.cuda())
    assert all(gpu.equal(a, b) for a, b in zip(plain, moved))
    for bad in (lambda t: t[:1], lambda t: t.double(), lambda t: t.cpu()):
        with pytest.raises(RuntimeError, match="saved-tensor hook"):
            grads(lambda t: t, bad)


def test_entry_points_in_place_and_with_every_output(gpu):
    """The C entry points: y and codes in one pass, y over x, the residual updated in place; dX over dY and
    dR over H in the backward pass."""
    R, K = 37, 1000
    x, r, w = case(R, K, np.float32)
    h = ref.stored(x, r)
    xd, rd, wd = to_dev(x), to_dev(r), to_dev(w)
    q = gpu.empty((R, K), dtype=gpu.uint8, device="cuda")
    s = gpu.empty((R, 8), device="cuda")
    L, st = tg.lib(), gpu.cuda.current_stream().cuda_stream
    assert L.rmsnorm_f16(R, K, xd.data_ptr(), K, rd.data_ptr(), K, 1, wd.data_ptr(), 0, EPS, rd.data_ptr(), K, xd.data_ptr(), K,
                         q.data_ptr(), K, s.data_ptr(), st) == 0
    assert np.array_equal(rd.cpu().numpy(), h)
    check_y(xd, h, w)
    check_codes(q, s, h, w)
    rng = np.random.default_rng(4)
    dy, dh = (0.1 * rng.standard_normal((R, K))).astype(np.float16), (0.1 * rng.standard_normal((R, K))).astype(np.float32)
    dx, bound, dw, size = ref.gradient(dy, h, w, EPS, dh)
    dyd, dhd, dwd = to_dev(dy), to_dev(dh), gpu.empty(K, dtype=gpu.float16, device="cuda")
    need = L.rmsnorm_f16_backward_workspace_bytes(R, K)
    ws = gpu.empty(need, dtype=gpu.uint8, device="cuda")
    assert L.rmsnorm_f16_backward(R, K, dyd.data_ptr(), K, rd.data_ptr(), K, 1, wd.data_ptr(), 0, EPS, dhd.data_ptr(), K,
                                  dyd.data_ptr(), K, rd.data_ptr(), K, dwd.data_ptr(), ws.data_ptr(), need, st) == 0
    tol = bound + np.abs(dx) * (ref.HALF16 + 2.0 ** -18) + ref.TINY16
    assert (np.abs(dyd.cpu().numpy() - dx) <= tol).all() and (np.abs(rd.cpu().numpy() - dx) <= bound + np.abs(dx) * 2.0 ** -18).all()
    assert (np.abs(dwd.cpu().numpy() - dw) <= size * 2.0 ** -17 + np.abs(dw) * ref.HALF16 + ref.TINY16).all()


def test_training_on_a_side_stream(gpu):
    """Forward and backward under another current stream than the default give the same bits."""
    x, r, w = case(300, 1000, np.float16)
    dy = to_dev(np.full((300, 1000), 0.25, dtype=np.float16))

    def step():
        leaves = [to_dev(t).requires_grad_() for t in (x, w, r)]
        y, h = tg.RmsNormFunction.apply(*leaves, EPS)
        return (y.detach(), *gpu.autograd.grad((y, h), leaves, (dy, dy)))

    plain = step()
    side = gpu.cuda.Stream()
    side.wait_stream(gpu.cuda.current_stream())
    with gpu.cuda.stream(side):
        other = step()
    side.synchronize()
    gpu.cuda.synchronize()
    assert all(gpu.equal(a, b) for a, b in zip(plain, other))
