"""MXFP4 on the GPU against float64 definitions (mx_reference): the quantiser and its inverse
code by code, both products on every kernel, ragged sizes, strides, alignments, special scales,
degenerate sizes, streams, graphs, and the autograd forms."""
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


def dev_matrix(codes, scale, pad=None):
    """Device copies; scale rows padded to `pad` bytes (default: 16-byte multiples, as the
    package allocates them), the padding filled with NaN scales."""
    R, kb = scale.shape
    width = -(-kb // 16) * 16 if pad is None else kb + pad
    s = np.full((R, width), 255, dtype=np.uint8)
    s[:, :kb] = scale
    return to_dev(codes), to_dev(s)[:, :kb]


def spread(rng, R, K, lo=-24, hi=15):
    """float16 values whose blocks span binary16's range, zeros and subnormals among them."""
    x = rng.standard_normal((R, K)) * 2.0 ** rng.integers(lo, hi, (R, K // 16 + 1)).repeat(16, 1)[:, :K]
    x[rng.random((R, K)) < 0.05] = 0.0
    x[rng.random((R, K)) < 0.01] = -0.0
    if R > 2:
        x[1] = 0.0
    return np.clip(x, -65504, 65504).astype(np.float16)


QUANT_SHAPES = [(1, 1), (1, 4096), (3, 31), (33, 32), (257, 130), (255, 1000), (300, 129), (64, 2056), (1000, 40)]


@pytest.mark.parametrize("shape", QUANT_SHAPES, ids=str)
def test_quant_and_dequant(gpu, shape):
    R, K = shape
    rng = np.random.default_rng(R * 10007 + K)
    x = spread(rng, R, K)
    xd = to_dev(x)
    q, s, qt, st = tg.mxfp4_quant(xd, "both")
    for name, (qq, ss) in {"rows": (q, s), "cols": (qt, st)}.items():
        ref_q, ref_s = mx.quant(x if name == "rows" else np.ascontiguousarray(x.T))
        assert np.array_equal(ss.cpu().numpy(), ref_s), name
        assert np.array_equal(qq.cpu().numpy(), ref_q), name
        one_q, one_s = tg.mxfp4_quant(xd, name)
        assert gpu.equal(one_q, qq) and gpu.equal(one_s, ss)
        k = K if name == "rows" else R
        v = tg.mxfp4_dequant(qq, ss, k)
        want = mx.to_half(mx.values(ref_q, ref_s)[:, :k])
        assert np.array_equal(v.cpu().numpy().view(np.uint16), want.view(np.uint16)), name


def test_quant_every_binary16_value(gpu):
    """Every finite binary16 magnitude as a block's maximum beside every midpoint of its grid."""
    bits = np.arange(0x7C00, dtype=np.uint16)
    top = bits.view(np.float16).astype(np.float64)
    e = np.where(top > 0, np.frexp(np.where(top > 0, top, 1))[1] - 3, 0)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 0.24, 0.26, 0.74, 0.76, 1.24, 1.26, 1.74, 1.76])
    x = np.zeros((len(bits), 32))
    x[:, 0] = top
    x[:, 1:16] = np.minimum(mids[None] * 2.0 ** e[:, None], top[:, None])
    x[:, 16:31] = -x[:, 1:16]
    x = x.astype(np.float16)
    q, s = tg.mxfp4_quant(to_dev(x))
    ref_q, ref_s = mx.quant(x)
    assert np.array_equal(s.cpu().numpy(), ref_s) and np.array_equal(q.cpu().numpy(), ref_q)


def test_dequant_every_code_and_scale(gpu):
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scale = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    v = tg.mxfp4_dequant(*dev_matrix(codes, scale), 512).cpu().numpy()
    want = mx.to_half(mx.values(codes, scale))
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(v), nan)
    assert np.array_equal(v[~nan].view(np.uint16), want[~nan].view(np.uint16))


def test_quant_nonfinite_and_strided(gpu):
    rng = np.random.default_rng(9)
    x = spread(rng, 70, 100, -4, 4)
    x[3, 5], x[40, 64], x[69, 99] = np.inf, np.nan, -np.inf
    for off, ld in ((0, 100), (1, 101), (3, 135)):
        buf = gpu.zeros(70 * ld + 8, dtype=gpu.float16, device="cuda")
        xd = buf[off:].as_strided((70, 100), (ld, 1))
        xd.copy_(to_dev(x))
        q, s, qt, st = tg.mxfp4_quant(xd, "both")
        for a, b, ref in ((q, s, mx.quant(x)), (qt, st, mx.quant(np.ascontiguousarray(x.T)))):
            assert np.array_equal(a.cpu().numpy(), ref[0]) and np.array_equal(b.cpu().numpy(), ref[1])
        assert gpu.isnan(tg.mxfp4_dequant(q, s, 100)[3, :32]).all()
    # strided and misaligned codes, scales and output through the C entry points
    L, st_ = tg.lib(), gpu.cuda.current_stream().cuda_stream
    qb = gpu.full((70, 67), 7, dtype=gpu.uint8, device="cuda")
    sb = gpu.full((70, 5), 9, dtype=gpu.uint8, device="cuda")
    xd = to_dev(x)
    assert L.mxfp4_quant(70, 100, xd.data_ptr(), 100, qb.data_ptr() + 1, 67, sb.data_ptr(), 5, None, 0, None, 0, st_) == 0
    gpu.cuda.synchronize()
    ref = mx.quant(x)
    got = qb.cpu().numpy()
    assert np.array_equal(got[:, 1:65], ref[0]) and (got[:, 0] == 7).all() and (got[:, 65:] == 7).all()
    assert np.array_equal(sb.cpu().numpy()[:, :4], ref[1]) and (sb[:, 4] == 9).all()
    out = gpu.full((70, 103), 3.0, dtype=gpu.float16, device="cuda")
    assert L.mxfp4_dequant(70, 100, qb.data_ptr() + 1, 67, sb.data_ptr(), 5, out.data_ptr() + 2, 103, st_) == 0
    gpu.cuda.synchronize()
    o, want = out.cpu().numpy(), mx.to_half(mx.values(*ref)[:, :100])
    assert np.array_equal(o[:, 1:101], want, equal_nan=True) and (o[:, 0] == 3).all() and (o[:, 101:] == 3).all()


# Sizes around the 16-, 128- and 256-wide tiles, the k-tiles of 32 and 128 and the scale groups of 512.
GEMM_SHAPES = [(1, 1, 1), (1, 16, 512), (2, 40, 33), (16, 17, 544), (17, 300, 2080), (33, 264, 1100), (64, 130, 96),
               (65, 257, 128), (128, 128, 1056), (300, 513, 640), (257, 255, 160), (520, 392, 4128),
               (130, 40, 1000)]
CONFIGS = [None, tg.MX_GENERIC, tg.MX_SKINNY, tg.MX_128, tg.MX_256, tg.MX_64]
CONFIGS_F16 = CONFIGS[:-1]  # no 64 x 128 tiles with binary16 A


def f16_case(M, N, K, seed, lo=116, hi=132):
    rng = np.random.default_rng(seed)
    a = (rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.02, 12, 1)).astype(np.float16)
    return a, *mx.random_matrix(rng, N, K, lo, hi)


@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: f"cfg{c}")
def test_gemm(gpu, cfg):
    for i, (M, N, K) in enumerate(GEMM_SHAPES):
        if cfg == tg.MX_SKINNY and M > tg.MX_SKINNY_ROWS:
            continue
        rng = np.random.default_rng(500 + i)
        A, sa = mx.random_matrix(rng, M, K, 100, 126)
        B, sb = mx.random_matrix(rng, N, K, 118, 140)
        for relu in (False, True):
            log(f"mxfp4 cfg {cfg} {M}x{N}x{K} relu={relu}")
            out = gpu.full((M, N + 3), 5.0, dtype=gpu.float16, device="cuda")
            tg.mxfp4_gemm(*dev_matrix(A, sa), *dev_matrix(B, sb), c=out[:, :N], relu=relu, cfg=cfg)
            gpu.cuda.synchronize()
            ref, tol = mx.product(mx.values(A, sa), mx.values(B, sb), relu)
            mx.check(out[:, :N].cpu().numpy(), ref, tol, f"cfg {cfg} {M}x{N}x{K}")
            assert (out[:, N:] == 5.0).all()


@pytest.mark.parametrize("cfg", CONFIGS_F16, ids=lambda c: f"cfg{c}")
def test_gemm_f16(gpu, cfg):
    for i, (M, N, K) in enumerate(GEMM_SHAPES):
        if cfg == tg.MX_SKINNY and M > tg.MX_SKINNY_ROWS:
            continue
        if cfg not in (None, tg.MX_GENERIC, tg.MX_SKINNY):
            K = -(-K // 8) * 8
        a, B, sb = f16_case(M, N, K, 700 + i)
        for relu in (False, True):
            log(f"f16 x mxfp4 cfg {cfg} {M}x{N}x{K} relu={relu}")
            out = gpu.full((M, N + 3), 5.0, dtype=gpu.float16, device="cuda")
            tg.mxfp4_gemm_f16(to_dev(a), *dev_matrix(B, sb), c=out[:, :N], relu=relu, cfg=cfg)
            gpu.cuda.synchronize()
            w = mx.to_half(mx.values(B, sb)[:, :K]).astype(np.float64)
            ref, tol = mx.product(a.astype(np.float64), w, relu)
            mx.check(out[:, :N].cpu().numpy(), ref, tol, f"cfg {cfg} {M}x{N}x{K}")
            assert (out[:, N:] == 5.0).all()


@pytest.mark.parametrize("cfg", CONFIGS[1:], ids=lambda c: f"cfg{c}")
def test_extreme_and_nan_scales(gpu, cfg):
    """Scales from the smallest to the largest that cancel in the product, products that leave
    binary16's range, zero codes beside them, NaN scales in single blocks."""
    M, N, K = 40, 48, 576
    rng = np.random.default_rng(31)
    A, sa = mx.random_matrix(rng, M, K, 0, 60)
    B, sb = mx.random_matrix(rng, N, K, 190, 254)
    sa[0], sb[0] = 0, 254
    sa[5, 3], sa[6, 17], sb[9, 0] = 255, 255, 255
    sa[7], A[7] = 254, 0
    ref, tol = mx.product(mx.values(A, sa), mx.values(B, sb))
    got = tg.mxfp4_gemm(*dev_matrix(A, sa), *dev_matrix(B, sb), cfg=cfg)
    mx.check(got.cpu().numpy(), ref, tol, "extreme scales")
    relu = tg.mxfp4_gemm(*dev_matrix(A, sa), *dev_matrix(B, sb), relu=True, cfg=cfg).cpu().numpy()
    assert (relu[5] == 0).all() and (relu[:, 9] == 0).all()
    if cfg not in CONFIGS_F16:
        return
    a, B, sb = f16_case(M, N, K, 32, 90, 145)
    B[3], sb[3] = 0, 254
    sb[11, 4], sb[12, 17] = 255, 255
    w = mx.to_half(mx.values(B, sb)[:, :K]).astype(np.float64)
    got = tg.mxfp4_gemm_f16(to_dev(a), *dev_matrix(B, sb), cfg=cfg).cpu().numpy()
    fine = np.isfinite(w).all(1)
    ref, tol = mx.product(a.astype(np.float64), w[fine])
    mx.check(got[:, fine], ref, tol, "weights over binary16's range")
    assert not np.isfinite(got[:, ~fine]).any() and np.isnan(got[:, [11, 12]]).all()


def test_block_sums_keep_float32_precision(gpu):
    """Large products that cancel beside small ones: the sum keeps what float32 keeps."""
    M, N, K = 32, 64, 128
    rng = np.random.default_rng(77)
    for cfg in CONFIGS[1:]:
        worst = 0.0
        for gap in (0, 4, 8, 12, 16, 20):
            A, sa = mx.random_matrix(rng, M, K, 127, 127)
            B, sb = mx.random_matrix(rng, N, K, 127, 127)
            A[:, 16:32] = A[:, :16] ^ 0x88      # block 1 is minus block 0
            B[:, 16:32] = B[:, :16]
            sa[:, :2] += gap
            ref, tol = mx.product(mx.values(A, sa), mx.values(B, sb))
            c = tg.mxfp4_gemm(*dev_matrix(A, sa), *dev_matrix(B, sb), cfg=cfg).cpu().numpy()
            worst = max(worst, mx.check(c, ref, tol, f"cfg {cfg} gap 2^{gap}"))
        log(f"cfg {cfg}: worst error / tolerance {worst:.3f}")


def test_unaligned_operands_take_the_generic_kernel(gpu):
    M, N, K = 70, 90, 200
    rng = np.random.default_rng(41)
    A, sa = mx.random_matrix(rng, M, K)
    B, sb = mx.random_matrix(rng, N, K)
    ref, tol = mx.product(mx.values(A, sa), mx.values(B, sb))

    def shifted(x, off, ld):
        buf = gpu.zeros(off + x.shape[0] * ld, dtype=gpu.uint8, device="cuda")
        v = buf[off:].as_strided(x.shape, (ld, 1))
        v.copy_(to_dev(x))
        return v

    for off, ldq, lds in ((1, 113, 7), (0, 112, 7), (16, 112, 16), (5, 130, 9)):
        c = tg.mxfp4_gemm(shifted(A, off, ldq), shifted(sa, off, lds), shifted(B, off, ldq), shifted(sb, off, lds))
        mx.check(c.cpu().numpy(), ref, tol, f"offset {off} strides {ldq} {lds}")
    w = mx.to_half(mx.values(B, sb)[:, :K]).astype(np.float64)
    cases = [(M, *f16_case(M, N, K, 42)[:1], off, ld) for M in (70, 300) for off, ld in ((1, 200), (0, 203), (8, 208))]
    for M, a, off, ld in cases:
        ref, tol = mx.product(a.astype(np.float64), w)
        buf = gpu.full((off + M * ld,), float("nan"), dtype=gpu.float16, device="cuda")
        ad = buf[off:].as_strided((M, K), (ld, 1))
        ad.copy_(to_dev(a))
        for kernel in (None, tg.MX_GENERIC):
            c = tg.mxfp4_gemm_f16(ad, *dev_matrix(B, sb), cfg=kernel)
            mx.check(c.cpu().numpy(), ref, tol, f"{M} rows of a at {off}, stride {ld}, kernel {kernel}")


def test_degenerate_sizes(gpu):
    q, s = tg.mxfp4_empty(5, 0, "cuda")
    r, t = tg.mxfp4_empty(3, 0, "cuda")
    assert (tg.mxfp4_gemm(q, s, r, t) == 0).all()
    a = gpu.empty((4, 0), dtype=gpu.float16, device="cuda")
    assert (tg.mxfp4_gemm_f16(a, r, t) == 0).all()
    e = gpu.empty((0, 64), dtype=gpu.float16, device="cuda")
    q0, s0, qt, st = tg.mxfp4_quant(e, "both")
    assert q0.shape == (0, 32) and s0.shape == (0, 2) and qt.shape == (64, 0) and st.shape == (64, 0)
    q, s = tg.mxfp4_quant(gpu.ones((3, 64), dtype=gpu.float16, device="cuda"))
    assert tg.mxfp4_gemm(q0, s0, q, s).shape == (0, 3) and tg.mxfp4_gemm(q, s, q0, s0).shape == (3, 0)
    assert tg.mxfp4_dequant(q0, s0, 64).shape == (0, 64)


def test_python_argument_checks(gpu):
    q, s = tg.mxfp4_quant(gpu.ones((4, 64), dtype=gpu.float16, device="cuda"))
    with pytest.raises(ValueError, match="belong together"):
        tg.mxfp4_gemm(q, s[:, :1], q, s)
    with pytest.raises(ValueError, match="inner dimensions"):
        tg.mxfp4_gemm(q, s, q[:, :16], s[:, :1])
    with pytest.raises(ValueError, match="inner dimensions"):
        tg.mxfp4_gemm_f16(gpu.ones((4, 32), dtype=gpu.float16, device="cuda"), q, s)
    with pytest.raises(ValueError, match="expected"):
        tg.mxfp4_gemm(q, s, q, s, c=gpu.empty((4, 5), dtype=gpu.float16, device="cuda"))
    with pytest.raises(ValueError, match="do not hold"):
        tg.mxfp4_dequant(q, s, 96)
    with pytest.raises(ValueError, match="dims"):
        tg.mxfp4_quant(gpu.ones((4, 64), dtype=gpu.float16, device="cuda"), "all")
    with pytest.raises(ValueError):
        tg.mxfp4_gemm(q.t(), s, q, s)


def test_deterministic_and_other_stream(gpu):
    rng = np.random.default_rng(12)
    for M in (8, 300):
        x = to_dev(spread(rng, M, 1000, -3, 3))
        w = to_dev(spread(rng, 200, 1000, -6, 0))
        wq = tg.mxfp4_quant(w)
        ref = tg.mxfp4_linear(x, *wq)
        ref16 = tg.mxfp4_gemm_f16(x, *wq)
        gpu.cuda.synchronize()
        side = gpu.cuda.Stream()
        outs = [gpu.empty((M, 200), dtype=gpu.float16, device="cuda") for _ in range(2)]
        xq = tg.mxfp4_quant(x, stream=side)
        tg.mxfp4_gemm(*xq, *wq, c=outs[0], stream=side)
        tg.mxfp4_gemm_f16(x, *wq, c=outs[1], stream=side)
        side.synchronize()
        assert gpu.equal(outs[0], ref) and gpu.equal(outs[1], ref16)


def test_graph_replays(gpu):
    """A linear layer's quantiser, products and inverse captured once, replayed on new inputs
    with eager work between the replays."""
    rng = np.random.default_rng(13)
    w = to_dev(spread(rng, 130, 640, -6, 0))
    wq = tg.mxfp4_quant(w)
    for M in (3, 140):
        x = gpu.zeros((M, 640), dtype=gpu.float16, device="cuda")
        tg.mxfp4_linear(x, *wq)
        side = gpu.cuda.Stream()
        side.wait_stream(gpu.cuda.current_stream())
        g = gpu.cuda.CUDAGraph()
        with gpu.cuda.graph(g, stream=side):
            q, s, qt, st = tg.mxfp4_quant(x, "both")
            y = tg.mxfp4_gemm(q, s, *wq, relu=True)
            z = tg.mxfp4_gemm_f16(x, *wq)
            v = tg.mxfp4_dequant(qt, st, M)
        for _ in range(4):
            x.copy_(to_dev(spread(rng, M, 640, -3, 3)))
            g.replay()
            gpu.cuda.synchronize()
            e = tg.mxfp4_quant(x, "both")
            assert gpu.equal(y, tg.mxfp4_gemm(*e[:2], *wq, relu=True))
            assert gpu.equal(z, tg.mxfp4_gemm_f16(x, *wq))
            assert gpu.equal(v, tg.mxfp4_dequant(*e[2:], M))


GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, -0.5, -1, -1.5, -2, -3, -4])


@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (37, 70, 100), (96, 130, 257)])
def test_linear_gradients(gpu, M, N, K):
    """Inputs on the grid quantise to themselves, so output and gradients are the plain
    linear layer's: exact but for the result's rounding, and equal to difference quotients."""
    rng = np.random.default_rng(M)
    x, w, dy = (rng.choice(GRID, sh) for sh in ((M, K), (N, K), (M, N)))
    xd, wd = (to_dev(v.astype(np.float16)).requires_grad_() for v in (x, w))
    y = tg.Mxfp4LinearFunction.apply(xd, wd)
    gx, gw = gpu.autograd.grad(y, (xd, wd), to_dev(dy.astype(np.float16)))
    for got, a, b in ((y.detach(), x, w), (gx, dy, w.T), (gw, dy.T, x.T)):
        ref, tol = mx.product(a, b)
        mx.check(got.cpu().numpy(), ref, tol)
    # d/dx[i, k] of sum(dy * y) by a step of the grid (y is linear there)
    i, k = M // 2, K // 3
    x2 = x.copy()
    x2[i, k] = 4.0 if x[i, k] <= 0 else -4.0
    y2 = tg.Mxfp4LinearFunction.apply(to_dev(x2.astype(np.float16)), wd.detach())
    diff = (y2.double() - y.detach().double()).cpu().numpy()
    quotient = float((dy[i] * diff[i]).sum() / (x2[i, k] - x[i, k]))
    slack = (np.abs(dy[i]) * 2 * (2.0 ** -11) * (np.abs(x) @ np.abs(w).T).max()).sum() / abs(x2[i, k] - x[i, k])
    assert abs(quotient - float(gx[i, k])) <= slack + 2.0 ** -10 * abs(float(gx[i, k]))


def test_linear_gradients_of_plain_values(gpu):
    """Off the grid: the three products of the step on operands quantised along each one's own
    inner dimension; broadcast and transposed upstream gradients."""
    M, N, K = 70, 96, 130
    rng = np.random.default_rng(6)
    x, w, dy = (rng.standard_normal(s).astype(np.float16) for s in ((M, K), (N, K), (M, N)))

    def q(v):
        v = np.ascontiguousarray(v)
        return mx.values(*mx.quant(v))[:, :v.shape[1]]

    xd, wd = to_dev(x).requires_grad_(), to_dev(w).requires_grad_()
    row = rng.standard_normal((1, N)).astype(np.float16)
    for d, up in ((dy, to_dev(dy)), (dy, to_dev(np.ascontiguousarray(dy.T)).t()), (np.repeat(row, M, 0), to_dev(row).expand(M, N))):
        y = tg.Mxfp4LinearFunction.apply(xd, wd)
        gx, gw = gpu.autograd.grad(y, (xd, wd), up)
        for got, a, b in ((y.detach(), q(x), q(w)), (gx, q(d), q(w.T)), (gw, q(d.T), q(x.T))):
            mx.check(got.cpu().numpy(), *mx.product(a, b))
    # one gradient wanted only, and a transposed input
    y = tg.Mxfp4LinearFunction.apply(xd, wd.detach())
    mx.check(gpu.autograd.grad(y, xd, to_dev(dy))[0].cpu().numpy(), *mx.product(q(dy), q(w.T)))
    wt = to_dev(np.ascontiguousarray(w.T)).t().requires_grad_()
    y = tg.Mxfp4LinearFunction.apply(xd.detach(), wt)
    mx.check(gpu.autograd.grad(y, wt, to_dev(dy))[0].cpu().numpy(), *mx.product(q(dy.T), q(x.T)))


@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (50, 96, 257), (130, 72, 100), (300, 77, 330)])
def test_weight_gradients(gpu, M, N, K):
    rng = np.random.default_rng(K)
    a, B, sb = f16_case(M, N, K, K, 118, 126)
    w = mx.values(B, sb)[:, :K]
    dy = rng.standard_normal((M, N)).astype(np.float16)
    xd = to_dev(a).requires_grad_()
    y = tg.Mxfp4WeightFunction.apply(xd, *dev_matrix(B, sb))
    gx, = gpu.autograd.grad(y, xd, to_dev(dy))
    mx.check(y.detach().cpu().numpy(), *mx.product(a.astype(np.float64), w))
    mx.check(gx.cpu().numpy(), *mx.product(dy.astype(np.float64), w.T))
    # y is linear in x: a difference quotient over a whole step is the gradient
    i, k = M - 1, K // 2
    a2 = a.copy()
    a2[i, k] += np.float16(4.0)
    y2 = tg.Mxfp4WeightFunction.apply(to_dev(a2), *dev_matrix(B, sb))
    h = float(a2[i, k]) - float(a[i, k])
    diff = (y2[i].double() - y.detach()[i].double()).cpu().numpy()
    quotient = float((dy[i].astype(np.float64) * diff).sum() / h)
    size = np.maximum(np.abs(a2[i].astype(np.float64)), np.abs(a[i].astype(np.float64))) @ np.abs(w).T
    assert abs(quotient - float(gx[i, k])) <= float((np.abs(dy[i]) * size).sum()) * 2.0 ** -10 / h + 2.0 ** -10 * abs(float(gx[i, k]))


@pytest.mark.parametrize("M,N,K", [(48, 8192, 8192), (4095, 4100, 1056)])
def test_large_sampled(gpu, M, N, K):
    """The default choice on large ragged outputs, whole sampled rows and columns."""
    rng = np.random.default_rng(N)
    A, sa = mx.random_matrix(rng, M, K, 118, 124)
    B, sb = mx.random_matrix(rng, N, K, 118, 124)
    c = tg.mxfp4_gemm(*dev_matrix(A, sa), *dev_matrix(B, sb)).cpu().numpy()
    a = mx.values(A, sa)
    a16 = a[:, :K].astype(np.float16)
    c16 = tg.mxfp4_gemm_f16(to_dev(a16), *dev_matrix(B, sb)).cpu().numpy()
    rows = np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, 6)]))
    cols = np.unique(np.concatenate([[0, N - 1], rng.integers(0, N, 6)]))
    b = mx.values(B[cols], sb[cols])
    mx.check(c[:, cols], *mx.product(a, b))
    mx.check(c16[:, cols], *mx.product(a, b))
    b = mx.values(B, sb)
    mx.check(c[rows], *mx.product(a[rows], b))
    mx.check(c16[rows], *mx.product(a[rows], b))


def test_strides_past_32_bits(gpu):
    """Row strides that put the last row past 2^32 bytes from the first."""
    M, N, K = 3, 40, 64
    rng = np.random.default_rng(55)
    B, sb = mx.random_matrix(rng, N, K, 120, 126)
    ld = (1 << 31) // 2 + 16
    buf = gpu.zeros(2 * ld + K, dtype=gpu.float16, device="cuda")
    a = rng.standard_normal((M, K)).astype(np.float16)
    ad = buf.as_strided((M, K), (ld, 1))
    ad.copy_(to_dev(a))
    assert tg.mxfp4_select_config(M, N, K, True, lda=ld) == tg.MX_SKINNY
    for cfg in (None, tg.MX_GENERIC):
        c = tg.mxfp4_gemm_f16(ad, *dev_matrix(B, sb), cfg=cfg)
        mx.check(c.cpu().numpy(), *mx.product(a.astype(np.float64), mx.values(B, sb)))
    q, s, qt, st = tg.mxfp4_quant(ad, "both")
    assert np.array_equal(q.cpu().numpy(), mx.quant(a)[0]) and np.array_equal(qt.cpu().numpy(), mx.quant(a.T.copy())[0])
    out = tg.mxfp4_dequant(q, s, K, out=ad)
    assert np.array_equal(out.cpu().numpy(), mx.to_half(mx.values(*mx.quant(a))))


def test_no_second_derivative(gpu):
    x = gpu.ones((4, 64), dtype=gpu.float16, device="cuda", requires_grad=True)
    w = gpu.ones((8, 64), dtype=gpu.float16, device="cuda", requires_grad=True)
    for y in (tg.Mxfp4LinearFunction.apply(x, w), tg.Mxfp4WeightFunction.apply(x, *tg.mxfp4_quant(w.detach()))):
        with pytest.raises(RuntimeError, match="second derivative"):
            gpu.autograd.grad(y.sum(), x, create_graph=True)


@pytest.mark.parametrize("form", ["linear", "weight"])
def test_captured_step(gpu, form):
    """Output and gradients captured once (leaves of the capture's own) and replayed on new
    inputs, with the eager step between the replays."""
    rng = np.random.default_rng(41)
    M, N, K = 100, 264, 200
    wq = tg.mxfp4_quant(to_dev(spread(rng, N, K, -6, 0)))

    def step(x, w, dy):
        if form == "linear":
            y = tg.Mxfp4LinearFunction.apply(x, w)
            return (y.detach(), *gpu.autograd.grad(y, (x, w), dy))
        y = tg.Mxfp4WeightFunction.apply(x, *wq)
        return (y.detach(), *gpu.autograd.grad(y, (x,), dy))

    def leaves():
        return [gpu.zeros(sh, dtype=gpu.float16, device="cuda").requires_grad_(grad)
                for sh, grad in (((M, K), True), ((N, K), True), ((M, N), False))]

    static = leaves()
    side = gpu.cuda.Stream()
    side.wait_stream(gpu.cuda.current_stream())
    with gpu.cuda.stream(side):
        step(*leaves())
    side.synchronize()
    g = gpu.cuda.CUDAGraph()
    with gpu.cuda.graph(g, stream=side):
        out = step(*static)
    for _ in range(4):
        eager = leaves()
        for s, e in zip(static, eager):
            v = to_dev(spread(rng, *s.shape, -3, 1))
            s.detach().copy_(v)
            e.detach().copy_(v)
        g.replay()
        gpu.cuda.synchronize()
        for got, ref in zip(out, step(*eager)):
            assert gpu.equal(got, ref)


def test_weight_of_many_rows(gpu):
    """More rows than the skinny kernel's launch holds take other tiles."""
    N = 16 * ((1 << 22) - 1) + 1
    codes = gpu.full((N, 16), 0x22, dtype=gpu.uint8, device="cuda")            # every value 1
    scale = gpu.full((N, 16), 127, dtype=gpu.uint8, device="cuda")[:, :1]
    x = gpu.full((1, 32), 0.5, dtype=gpu.float16, device="cuda")
    scale[-1] = 128
    for y in (tg.mxfp4_gemm_f16(x, codes, scale), tg.mxfp4_gemm(*tg.mxfp4_quant(x), codes, scale)):
        assert bool((y[:, :-1] == 16).all()) and y[0, -1].item() == 32


def test_poisoned_copies(gpu):
    """On the build that fills every LDS copy's destination with NaN bytes first, each kernel's
    result stays the same bit for bit: no fragment or scale is read before its copy landed."""
    rng = np.random.default_rng(43)
    D = tg.debugfill_lib()
    for M, N, K in ((64, 130, 96), (130, 264, 2080), (300, 520, 1100), (520, 264, 4128)):
        x = to_dev(spread(rng, M, K, -3, 3))
        xq, wq = tg.mxfp4_quant(x), tg.mxfp4_quant(to_dev(spread(rng, N, K, -6, 0)))
        for cfg in CONFIGS:
            if cfg == tg.MX_SKINNY and M > tg.MX_SKINNY_ROWS:
                continue
            log(f"poisoned copies {M}x{N}x{K} kernel {cfg}")
            assert gpu.equal(tg.mxfp4_gemm(*xq, *wq, cfg=cfg, library=D), tg.mxfp4_gemm(*xq, *wq, cfg=cfg))
            if cfg != tg.MX_64 and (K % 8 == 0 or cfg in (None, tg.MX_GENERIC, tg.MX_SKINNY)):
                assert gpu.equal(tg.mxfp4_gemm_f16(x, *wq, cfg=cfg, library=D), tg.mxfp4_gemm_f16(x, *wq, cfg=cfg))
