"""An expert layer's operators on the GPU against their definitions (expert_reference): sorting exactly,
rows out and back, the products bit for bit on operands whose float32 sums are exact (every kernel,
form, ragged group and stride, on the product build and on the one that poisons every LDS copy's
destination) and inside their rounding bound on normal ones, gradients, the whole layer, streams and
graphs."""
import numpy as np
import pytest

import expert_reference as ref
from gpu_util import to_dev, torch_cuda

import tiled_dense_gemm_04_amd as tg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = torch_cuda()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tg.lib()
    return torch


def some_ids(rng, T, k, E, dropped=0.0, dtype=np.int64):
    """Distinct experts per token where there are enough, some liked more; dropped slots of several kinds."""
    score = rng.standard_normal((T, max(E, k))) + rng.standard_normal(max(E, k))
    ids = np.argsort(-score, axis=1)[:, :k] % E
    out = rng.random((T, k)) < dropped
    ids[out] = rng.choice([-1, E, E + 7, -(2 ** 31), 2 ** 31 - 1], out.sum())
    return np.ascontiguousarray(ids.astype(dtype))


def check_sort(plan, ids, E):
    for got, want, name in zip(plan, ref.sort(ids, E), plan._fields):
        assert np.array_equal(got.cpu().numpy(), want), name


# Sizes around the 64-slot steps, the chunks of 512 and 2048 slots, the limit of one launch (8192) and that
# of 256 chunks of 2048.
SORTS = [(0, 2, 4), (1, 1, 1), (1, 8, 8), (7, 3, 5), (64, 1, 64), (65, 1, 3), (255, 1, 2), (257, 1, 9), (100, 6, 60), (513, 8, 64),
         (1000, 4, 1024), (4097, 1, 1), (8191, 8, 256), (512, 1, 6), (2048, 4, 33), (2731, 3, 12), (65536, 1, 7), (262145, 2, 40), (65537, 1, 7), (10923, 6, 60), (20001, 5, 1024),
         (140000, 2, 128)]


@pytest.mark.parametrize("shape", SORTS, ids=str)
def test_sort(gpu, shape):
    T, k, E = shape
    rng = np.random.default_rng(T * 31 + E)
    for dropped, dtype in ((0.0, np.int64), (0.2, np.int32), (1.0, np.int64)):
        ids = some_ids(rng, T, k, E, dropped, dtype)
        check_sort(tg.expert_sort(to_dev(ids), E), ids, E)
    ids = np.full((T, k), E - 1, dtype=np.int32)  # all of them one expert's
    check_sort(tg.expert_sort(to_dev(ids), E), ids, E)


def test_sort_wide_ids_and_strides(gpu):
    rng = np.random.default_rng(1)
    ids = some_ids(rng, 300, 4, 16, 0.1)
    ids[0, 0], ids[1, 1], ids[2, 2] = 2 ** 32, 2 ** 32 + 3, -(2 ** 40)  # not 0, 3 or any other in 64 bits
    check_sort(tg.expert_sort(to_dev(ids), 16), ids, 16)
    wide = gpu.full((300, 9), 5, dtype=gpu.int64, device="cuda")
    wide[:, 3:7] = to_dev(ids)
    check_sort(tg.expert_sort(wide[:, 3:7], 16), ids, 16)
    big = some_ids(rng, 30000, 3, 20, 0.1, np.int32)
    wide = gpu.full((30000, 5), 5, dtype=gpu.int32, device="cuda")
    wide[:, 1:4] = to_dev(big)
    check_sort(tg.expert_sort(wide[:, 1:4], 20), big, 20)


def row_case(T, k, E, H, dropped, seed=0):
    rng = np.random.default_rng(seed + T * 7 + H)
    ids = some_ids(rng, T, k, E, dropped)
    x = rng.standard_normal((T, H)).astype(np.float16)
    y = rng.standard_normal((T * k, H)).astype(np.float16)
    w = rng.random((T, k)).astype(np.float32)
    return ids, x, y, w


ROWS = [(1, 1, 1, 1), (3, 2, 4, 7), (5, 3, 4, 8), (16, 2, 8, 4096), (33, 8, 64, 130), (100, 6, 60, 1001), (257, 5, 16, 264),
        (700, 4, 9, 2056), (2, 9, 12, 20000)]


def check_combine(out, y, place, w, k):
    want, size = ref.combine(y, place, w)
    # k products and k sums in float32, one rounding
    assert (np.abs(out.cpu().numpy() - want) <= np.abs(want) * ref.HALF16 + ref.TINY16 + 2 * k * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("shape", ROWS, ids=str)
def test_gather_and_combine(gpu, shape):
    T, k, E, H = shape
    for dropped in (0.0, 0.3, 1.0):
        ids, x, y, w = row_case(T, k, E, H, dropped)
        plan = tg.expert_sort(to_dev(ids), E)
        offsets, _, place = ref.sort(ids, E)
        base = np.full((T * k, H), 3.0, dtype=np.float16)
        out = to_dev(base)
        assert tg.expert_gather(to_dev(x), plan, out=out) is out
        assert np.array_equal(out.cpu().numpy(), ref.gather(x, place, base))  # rows behind the last as they were
        zero = tg.expert_gather(to_dev(x), plan, zero_rest=True)
        assert np.array_equal(zero.cpu().numpy(), ref.gather(x, place, np.zeros_like(base)))
        # rows that no slot has hold NaN: they are not read
        y[offsets[-1]:] = np.nan
        check_combine(tg.expert_combine(to_dev(y), plan, to_dev(w)), y, place, w, k)
        check_combine(tg.expert_combine(to_dev(y), plan), y, place, None, k)
        w16 = w.astype(np.float16)
        check_combine(tg.expert_combine(to_dev(y), plan, to_dev(w16)), y, place, w16, k)


def test_rows_of_any_stride_and_place(gpu):
    """Strided and misaligned rows; memory around them untouched; places outside the rows are skipped."""
    ids, x, y, w = row_case(50, 3, 6, 203, 0.2)
    plan = tg.expert_sort(to_dev(ids), 6)
    _, _, place = ref.sort(ids, 6)
    xb = gpu.zeros((50, 210), dtype=gpu.float16, device="cuda")
    xb[:, 3:206] = to_dev(x)
    ob = gpu.full((150, 211), 9.0, dtype=gpu.float16, device="cuda")
    tg.expert_gather(xb[:, 3:206], plan, out=ob[:, 5:208])
    assert np.array_equal(ob[:, 5:208].cpu().numpy(), ref.gather(x, place, np.full((150, 203), 9.0, dtype=np.float16)))
    assert (ob[:, :5] == 9).all() and (ob[:, 208:] == 9).all()
    yb = gpu.zeros((150, 209), dtype=gpu.float16, device="cuda")
    yb[:, 1:204] = to_dev(y)
    cb = gpu.full((50, 205), 4.0, dtype=gpu.float16, device="cuda")
    tg.expert_combine(yb[:, 1:204], plan, to_dev(w), out=cb[:, 1:204])
    check_combine(cb[:, 1:204], y, place, w, 3)
    assert (cb[:, 0] == 4).all() and (cb[:, 204:] == 4).all()
    odd = place.copy()
    odd[0], odd[1, 0], odd[2, 2] = 150, -7, 2 ** 31 - 1
    bad = tg.ExpertOrder(plan.offsets, plan.order, to_dev(odd))
    inside = np.where((odd >= 0) & (odd < 150), odd, -1)
    out = gpu.full((150, 203), 9.0, dtype=gpu.float16, device="cuda")
    tg.expert_gather(to_dev(x), bad, out=out)
    assert np.array_equal(out.cpu().numpy(), ref.gather(x, inside, np.full((150, 203), 9.0, dtype=np.float16)))
    check_combine(tg.expert_combine(to_dev(y), bad, to_dev(w)), y, inside, w, 3)


def test_combine_infinite_and_nan(gpu):
    ids, _, y, w = row_case(20, 2, 4, 64, 0.0)
    _, _, place = ref.sort(ids, 4)
    plan = tg.expert_sort(to_dev(ids), 4)
    y[place[3, 0], 5], y[place[4, 1], 6] = np.inf, np.nan
    w[5, 0] = np.inf
    out = tg.expert_combine(to_dev(y), plan, to_dev(w)).cpu().numpy()
    with np.errstate(all="ignore"):
        want = ref.combine(y, place, w)[0]
    assert np.array_equal(np.isnan(out), np.isnan(want)) and np.array_equal(np.isinf(out), np.isinf(want))


@pytest.mark.parametrize("shape", ROWS, ids=str)
def test_row_gradients(gpu, shape):
    T, k, E, H = shape
    for dropped, wtype in ((0.0, np.float32), (0.3, np.float16)):
        ids, x, y, w = row_case(T, k, E, H, dropped, seed=5)
        w = w.astype(wtype)
        rng = np.random.default_rng(8)
        dxs, dout = rng.standard_normal((T * k, H)).astype(np.float16), rng.standard_normal((T, H)).astype(np.float16)
        offsets, _, place = ref.sort(ids, E)
        plan = tg.expert_sort(to_dev(ids), E)
        xl = to_dev(x).requires_grad_()
        xs = tg.ExpertGatherFunction.apply(xl, *plan)
        assert np.array_equal(xs.detach().cpu().numpy(), ref.gather(x, place, np.zeros((T * k, H), dtype=np.float16)))
        dx, = gpu.autograd.grad(xs, xl, to_dev(dxs))
        check_combine(dx, dxs, place, None, k)
        yl, wl = to_dev(y).requires_grad_(), to_dev(w).requires_grad_()
        out = tg.ExpertCombineFunction.apply(yl, wl, *plan)
        check_combine(out.detach(), y, place, w, k)
        dy, dw = gpu.autograd.grad(out, (yl, wl), to_dev(dout))
        want = np.zeros((T * k, H))
        kept = place >= 0
        want[place[kept]] = (w.astype(np.float64)[..., None] * dout.astype(np.float64)[:, None])[kept]
        got = dy.cpu().numpy()
        assert (np.abs(got - want) <= np.abs(want) * (ref.HALF16 + 2.0 ** -24) + ref.TINY16).all()
        assert (got[offsets[-1]:] == 0).all()
        rows, d = ref.slots(y, place), dout.astype(np.float64)[:, None]
        want, size = (rows * d).sum(2), np.abs(rows * d).sum(2)
        # a lane adds H / 64 products, six more additions join the lanes
        tol = size * (H / 64 + 8 + 7) * 2.0 ** -24 + (0 if wtype == np.float32 else 1) * (np.abs(want) * ref.HALF16 + ref.TINY16)
        assert (np.abs(dw.cpu().numpy() - want) <= tol).all()
        # one of the two alone
        one, = gpu.autograd.grad(tg.ExpertCombineFunction.apply(yl, to_dev(w), *plan), yl, to_dev(dout))
        two, = gpu.autograd.grad(tg.ExpertCombineFunction.apply(to_dev(y), wl, *plan), wl, to_dev(dout))
        assert gpu.equal(one, dy) and gpu.equal(two, dw)
        plain, = gpu.autograd.grad(tg.ExpertCombineFunction.apply(yl, None, *plan), yl, to_dev(dout))
        assert np.array_equal(plain.cpu().numpy(), ref.gather(dout, place, np.zeros((T * k, H), dtype=np.float16)))


# ------------------------------------------------------------------ products
def test_every_row_end(gpu):
    """Rows that end in every place of a chunk of eight, up to one chunk and past it."""
    for H in range(2, 18):
        test_gather_and_combine(gpu, (37, 3, 5, H))
        test_row_gradients(gpu, (37, 3, 5, H))


def small_ints(rng, *shape):
    """Integers of -2 .. 2: any sum of up to 2^22 products of two is exact in float32."""
    return rng.integers(-2, 3, shape).astype(np.float16)


def groups(counts, tail=0):
    o = np.concatenate([[0], np.cumsum(counts)])
    return o.astype(np.int32), int(o[-1]) + tail


# Groups around the tiles of 32, 128 and 256 rows, empty ones, one for all, rows behind the last.
GROUPS = {"one_row": groups([1]), "empty_first": groups([0, 5, 0, 1], 3), "ragged": groups([33, 1, 0, 129, 31, 64], 5),
          "all_in_one": groups([0, 0, 300, 0]), "none": groups([0, 0, 0], 40), "tiles": groups([256, 128, 32]),
          "wide": groups([257, 300, 511], 1),
          "many": groups(np.random.default_rng(3).integers(0, 4, 200), 9),
          "rounds": groups([900, 700, 3000, 129, 255]),
          "long": groups([5000, 40, 700]),
          "most": groups(np.random.default_rng(4).integers(0, 2, 1024), 2)}
SIZES = [(8, 8), (40, 64), (264, 72), (136, 520), (520, 1000)]   # N, K: the tiles' edges, k-tiles of 32 and 64
ODD = [(1, 1), (129, 65), (258, 131)]
FORMS = ["nt", "nn", "tn"]
CONFIGS = [None, tg.EXPERT_GENERIC, tg.EXPERT_32, tg.EXPERT_128, tg.EXPERT_256, tg.EXPERT_TILES, tg.EXPERT_64]
ROWS_ONLY = (tg.EXPERT_32, tg.EXPERT_64)   # kernels that the weights' form does not have


def stack_with_pad(b, pad, gap):
    """A strided device stack: rows padded by `pad`, matrices `gap` elements apart beyond their rows."""
    torch = torch_cuda()
    E, r, c = b.shape
    ld, st = c + pad, r * (c + pad) + gap
    buf = torch.full((E * st + 8,), float("nan"), dtype=torch.float16, device="cuda")
    view = buf.as_strided((E, r, c), (st, ld, 1))
    view.copy_(to_dev(b))
    return view


def run_product(form, a, b, offsets, N, cfg, relu=False, zero_rest=False, library=None, pad=0, gap=0):
    torch = torch_cuda()
    if form == "tn":
        c = torch.full((len(offsets) - 1, a.shape[1], N), float("nan"), dtype=torch.float16, device="cuda")
        tg.expert_gemm_f16_tn(to_dev(a), to_dev(b), to_dev(offsets), c, cfg=cfg, library=library)
    else:
        c = torch.full((len(a), N), 7.0, dtype=torch.float16, device="cuda")
        tg.expert_gemm_f16(to_dev(a), stack_with_pad(b, pad, gap), to_dev(offsets), c, relu=relu, trans_b=form == "nt",
                           zero_rest=zero_rest, cfg=cfg, library=library)
    return c.cpu().numpy()


def exact_product(form, rng, offsets, rows, N, K, cfg, **kw):
    a = small_ints(rng, rows, K)
    if form == "tn":
        b = small_ints(rng, rows, N)
        return run_product(form, a, b, offsets, N, cfg, library=kw.get("library")), ref.to_half(ref.products_tn(a, b, offsets))
    E = len(offsets) - 1
    b = small_ints(rng, E, N, K) if form == "nt" else small_ints(rng, E, K, N)
    rest = 0.0 if kw.get("zero_rest") else 7.0
    base = np.full((rows, N), 7.0)
    base[int(offsets[-1]):] = rest
    want, _ = ref.products(a, b, offsets, form == "nt", base)
    if kw.get("relu"):
        for lo, hi in ref.clamped(offsets, rows):
            want[lo:hi] = np.maximum(want[lo:hi], 0)
    return run_product(form, a, b, offsets, N, cfg, **kw), ref.to_half(want)


@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: f"cfg{c}")
@pytest.mark.parametrize("form", FORMS)
def test_products_exact(gpu, form, cfg):
    if form == "tn" and cfg in ROWS_ONLY:
        pytest.skip("not a kernel of this form")
    rng = np.random.default_rng(11)
    sizes = SIZES if cfg not in (None, tg.EXPERT_GENERIC) else SIZES + ODD
    for name, (offsets, rows) in GROUPS.items():
        for i, (N, K) in enumerate(sizes):
            if name == "most" and N * K > 3000 or name == "rounds" and N * K < 3000:
                continue
            print(f"{form} cfg {cfg} {name} {rows} rows N {N} K {K}", flush=True)
            if form == "nn" and cfg not in (None, tg.EXPERT_GENERIC):
                K += 3  # (K is then a contiguous dimension of A alone)
                K -= K % 8
            got, want = exact_product(form, rng, offsets, rows, N, K, cfg, relu=i % 2 == 1, zero_rest=i % 3 == 1)
            assert np.array_equal(got, want), (name, N, K)


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("counts, N", [([300, 0, 45, 129], 520), ([3000, 1400, 257], 1000), ([600, 520, 300, 129, 260], 2440),
                                       ([2000, 2100, 1700, 1000, 1500], 2056)], ids=lambda v: str(v))
def test_products_last_round_in_halves(gpu, form, counts, N):
    """Lists of tiles whose last round is of halves: all of one, after a round of small tiles, edges among them,
    and after a round of big tiles (quarters and edges)."""
    offsets, rows = groups(counts, 5)
    got, want = exact_product(form, np.random.default_rng(13), offsets, rows, N, 72, tg.EXPERT_TILES, relu=True,
                              zero_rest=True)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("form", FORMS)
def test_products_debug_fill(gpu, form):
    """The build that fills every LDS copy's destination with NaN first: no read before its copy."""
    rng = np.random.default_rng(12)
    for cfg in CONFIGS[2:]:
        if form == "tn" and cfg in ROWS_ONLY:
            continue
        for name in ("ragged", "wide", "empty_first", "long"):
            offsets, rows = GROUPS[name]
            for N, K in ((264, 72), (136, 520), (8, 8)):
                print(f"{form} cfg {cfg} {name} N {N} K {K}", flush=True)
                got, want = exact_product(form, rng, offsets, rows, N, K, cfg, library=tg.debugfill_lib())
                assert np.array_equal(got, want), (cfg, name, N, K)


def test_products_strides_and_alignment(gpu):
    rng = np.random.default_rng(13)
    offsets, rows = GROUPS["ragged"]
    for form in ("nt", "nn"):
        for pad, gap in ((8, 16), (3, 1), (0, 4), (16, 0)):
            for N, K in ((136, 200), (70, 72)):
                got, want = exact_product(form, rng, offsets, rows, N, K, None, pad=pad, gap=gap)
                assert np.array_equal(got, want), (form, pad, gap)
    # A, C and the offsets at odd places, C's rows apart: only the rows and columns asked for are written
    E, N, K = len(offsets) - 1, 130, 64
    a, b = small_ints(rng, rows, K), small_ints(rng, E, N, K)
    want = ref.to_half(ref.products(a, b, offsets, True, np.full((rows, N), 5.0))[0])
    for a_off, a_ld, c_off, c_ld in ((0, 64, 0, 136), (8, 72, 3, 137), (1, 65, 8, 144), (0, 64, 1, 130)):
        ab = gpu.zeros(rows * a_ld + 16, dtype=gpu.float16, device="cuda")
        av = ab[a_off:].as_strided((rows, K), (a_ld, 1))
        av.copy_(to_dev(a))
        cb = gpu.full((rows * c_ld + 16,), 5.0, dtype=gpu.float16, device="cuda")
        cv = cb[c_off:].as_strided((rows, N), (c_ld, 1))
        tg.expert_gemm_f16(av, to_dev(b), to_dev(np.concatenate([[9], offsets]).astype(np.int32))[1:], cv)
        assert np.array_equal(cv.cpu().numpy(), want)
        flat = cb.cpu().numpy()
        inside = np.zeros(flat.size, dtype=bool)
        inside[(c_off + np.arange(rows)[:, None] * c_ld + np.arange(N)).ravel()] = True
        assert (flat[~inside] == 5).all()
    # one matrix for all experts (stride 0), and a stack of results with gaps
    shared = to_dev(b[0]).expand(E, N, K)
    got = tg.expert_gemm_f16(to_dev(a), shared, to_dev(offsets), to_dev(np.full((rows, N), 5.0, dtype=np.float16)))
    want = ref.to_half(ref.products(a, np.repeat(b[:1], E, 0), offsets, True, np.full((rows, N), 5.0))[0])
    assert np.array_equal(got.cpu().numpy(), want)
    x, y = small_ints(rng, rows, 24), small_ints(rng, rows, 40)
    cb = gpu.full((E, 26, 43), 5.0, dtype=gpu.float16, device="cuda")
    tg.expert_gemm_f16_tn(to_dev(x), to_dev(y), to_dev(offsets), cb[:, :24, :40])
    assert np.array_equal(cb[:, :24, :40].cpu().numpy(), ref.to_half(ref.products_tn(x, y, offsets)))
    assert (cb[:, 24:] == 5).all() and (cb[:, :, 40:] == 5).all()


def test_offsets_outside_the_rows_are_clamped(gpu):
    rng = np.random.default_rng(14)
    offsets = np.array([-5, 3, 3, 40, 2 ** 31 - 1], dtype=np.int32)
    for cfg in CONFIGS:
        for form in FORMS:
            if form == "tn" and cfg in ROWS_ONLY:
                continue
            got, want = exact_product(form, rng, offsets, 70, 136, 64, cfg)
            assert np.array_equal(got, want), (cfg, form)


def test_empty_inner_dimension(gpu):
    offsets = to_dev(np.array([0, 2, 4], dtype=np.int32))
    c = gpu.full((6, 16), 3.0, dtype=gpu.float16, device="cuda")
    a = gpu.empty((6, 0), dtype=gpu.float16, device="cuda")
    tg.expert_gemm_f16(a, gpu.empty((2, 16, 0), dtype=gpu.float16, device="cuda"), offsets, c)
    assert (c[:4] == 0).all() and (c[4:] == 3).all()
    assert tg.expert_gemm_f16(gpu.empty((0, 8), dtype=gpu.float16, device="cuda"),
                              gpu.ones((2, 16, 8), dtype=gpu.float16, device="cuda"), offsets).shape == (0, 16)
    none = gpu.zeros(3, dtype=gpu.int32, device="cuda")
    d = tg.expert_gemm_f16_tn(gpu.empty((0, 24), dtype=gpu.float16, device="cuda"),
                              gpu.empty((0, 16), dtype=gpu.float16, device="cuda"), none)
    assert d.shape == (2, 24, 16) and (d == 0).all()


@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: f"cfg{c}")
def test_products_normal(gpu, cfg):
    """Normal operands inside the rounding bound, with ReLU and infinities."""
    rng = np.random.default_rng(15)
    offsets, rows = groups([130, 0, 300, 7, 64], 4)
    N, K = 392, 1032
    a = rng.standard_normal((rows, K)).astype(np.float16)
    b = (rng.standard_normal((5, N, K)) / 32).astype(np.float16)
    want, size = ref.products(a, b, offsets, True, np.zeros((rows, N)))
    got = run_product("nt", a, b, offsets, N, cfg, zero_rest=True)
    assert (np.abs(got - want) <= ref.product_bound(want, size, K)).all()
    relu = run_product("nt", a, b, offsets, N, cfg, relu=True, zero_rest=True)
    assert np.array_equal(relu, np.where(got > 0, got, np.float16(0)))
    assert np.array_equal(run_product("nn", a, np.ascontiguousarray(b.transpose(0, 2, 1)), offsets, N, cfg, zero_rest=True), got)
    if cfg not in ROWS_ONLY:
        dc = rng.standard_normal((rows, N)).astype(np.float16)
        got = run_product("tn", dc, a, offsets, K, cfg)
        want = ref.products_tn(dc, a, offsets)
        size = ref.products_tn(np.abs(dc), np.abs(a), offsets)
        assert (np.abs(got - want) <= ref.product_bound(want, size, 300)).all()
    # a NaN or an infinity stays in its row (and, over the rows, in its expert)
    a[140, 3], a[500, 0] = np.nan, np.inf
    dirty = run_product("nt", a, b, offsets, N, cfg, zero_rest=True)
    assert np.isnan(dirty[140]).all() and not np.isfinite(dirty[500]).any()
    keep = np.ones(rows, dtype=bool)
    keep[[140, 500]] = False
    clean = ref.products(a[keep], b, np.array([0, 130, 130, 429, 436, 499]), True, np.zeros((rows - 2, N)))[0]
    assert np.isfinite(dirty[keep]).all() and np.abs(dirty[keep] - clean).max() < 0.1


def test_large_offsets_in_a_long_buffer(gpu):
    """Rows and weights beyond 2^31 elements: sums of ones."""
    rows, K, N = 70000, 40960, 16
    a = gpu.zeros((rows, K), dtype=gpu.float16, device="cuda")   # 5.7 GB
    a[-300:, -8:] = 1
    b = gpu.zeros((2, N, K), dtype=gpu.float16, device="cuda")
    b[1] = 2
    offsets = to_dev(np.array([0, 69000, rows], dtype=np.int32))
    for cfg in CONFIGS:
        c = tg.expert_gemm_f16(a, b, offsets, cfg=cfg)
        assert (c[:-300] == 0).all() and (c[-300:] == 16).all()
    d = tg.expert_gemm_f16_tn(c, a, offsets)
    assert (d[0] == 0).all() and (d[1, :, :-8] == 0).all() and (d[1, :, -8:] == 4800).all()
    ids = gpu.arange(rows, device="cuda", dtype=gpu.int32).remainder(2).view(rows, 1)
    plan = tg.expert_sort(ids, 2)
    xs = tg.expert_gather(a, plan)
    assert int((xs[:, -1] == 1).sum()) == 300 and (xs[34850:35000, -1] == 1).all() and (xs[-150:, -1] == 1).all()
    assert gpu.equal(tg.expert_combine(xs, plan), a)


def test_product_gradients(gpu):
    rng = np.random.default_rng(16)
    for offsets, rows in (groups([40, 0, 200, 3], 5), groups([300, 10])):
        for N, K in ((136, 264), (65, 33)):
            E = len(offsets) - 1
            a, b, dc = small_ints(rng, rows, K), small_ints(rng, E, N, K), small_ints(rng, rows, N)
            al, bl = to_dev(a).requires_grad_(), to_dev(b).requires_grad_()
            c = tg.ExpertGemmFunction.apply(al, bl, to_dev(offsets))
            assert np.array_equal(c.detach().cpu().numpy(), ref.to_half(ref.products(a, b, offsets, True, np.zeros((rows, N)))[0]))
            da, db = gpu.autograd.grad(c, (al, bl), to_dev(dc))
            assert np.array_equal(da.cpu().numpy(), ref.to_half(ref.products(dc, b, offsets, False, np.zeros((rows, K)))[0]))
            assert np.array_equal(db.cpu().numpy(), ref.to_half(ref.products_tn(dc, a, offsets)))
            with pytest.raises(RuntimeError, match="second derivative"):
                gpu.autograd.grad(tg.ExpertGemmFunction.apply(al, bl, to_dev(offsets)).sum(), al, create_graph=True)
            # a broadcast gradient, and only one of the two
            ones = gpu.ones((), dtype=gpu.float16, device="cuda").expand(rows, N)
            da, = gpu.autograd.grad(tg.ExpertGemmFunction.apply(al, bl.detach(), to_dev(offsets)), al, ones)
            one = np.ones((rows, N), dtype=np.float16)
            assert np.array_equal(da.cpu().numpy(), ref.to_half(ref.products(one, b, offsets, False, np.zeros((rows, K)))[0]))


def test_broadcast_weight_gradient(gpu):
    """One matrix expanded over the experts, and one row expanded over a matrix: gradients are summed."""
    rng = np.random.default_rng(18)
    offsets, rows = groups([40, 7, 90])
    a, dc = small_ints(rng, rows, 64), small_ints(rng, rows, 40)
    one = small_ints(rng, 40, 64)
    w = to_dev(one).requires_grad_()
    c = tg.ExpertGemmFunction.apply(to_dev(a), w.expand(3, 40, 64), to_dev(offsets))
    assert np.array_equal(c.detach().cpu().numpy(), ref.to_half(a.astype(np.float64) @ one.T.astype(np.float64)))
    dw, = gpu.autograd.grad(c, w, to_dev(dc))
    each = ref.products_tn(dc, a, offsets)
    assert np.abs(dw.cpu().numpy() - each.sum(0)).max() <= 2 * np.abs(each).sum(0).max() * ref.HALF16
    row = to_dev(one[0]).requires_grad_()
    c = tg.ExpertGemmFunction.apply(to_dev(a), row.expand(3, 40, 64), to_dev(offsets))
    assert np.array_equal(c.detach().cpu().numpy(), ref.to_half(np.repeat(a.astype(np.float64) @ one[:1].T.astype(np.float64), 40, 1)))


# ------------------------------------------------------------------ together
def layer_inputs(T, k, E, H, F, seed, dropped=0.1):
    rng = np.random.default_rng(seed)
    ids = some_ids(rng, T, k, E, dropped)
    x = rng.standard_normal((T, H)).astype(np.float16)
    r = rng.standard_normal((T, H)).astype(np.float16)
    w = (1 + 0.1 * rng.standard_normal(H)).astype(np.float16)
    gate = rng.random((T, k)).astype(np.float32)
    up = (rng.standard_normal((E, F, H)) / np.sqrt(H)).astype(np.float16)
    down = (rng.standard_normal((E, H, F)) / np.sqrt(F)).astype(np.float16)
    return [to_dev(t) for t in (ids, x, r, w, gate, up, down)]


def layer(ids, x, r, w, gate, up, down, stream=None):
    y, h = tg.rmsnorm(x, w, r, stream=stream)
    plan = tg.expert_sort(ids, len(up), stream=stream)
    xs = tg.expert_gather(y, plan, stream=stream)
    inner = tg.expert_gemm_f16(xs, up, plan.offsets, relu=True, stream=stream)
    return tg.expert_combine(tg.expert_gemm_f16(inner, down, plan.offsets, stream=stream), plan, gate, stream=stream), h


def layer_in_float64(torch, ids, x, r, w, gate, up, down, open_=None):
    """The layer's output for float64 leaves on the CPU (differentiable). ``open_``: which values of the
    sorted inner rows pass ReLU, instead of the sign computed here. A gradient jumps where that sign
    turns: with errors of 2^-11 of a value's spread about 1e-4 of the values turn, each by all of its
    gradient, which is sqrt(1e-4) = 1e-2 of the gradient's norm, and no error of the gradient's
    computation."""
    h = x + r
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * w
    out, row = torch.zeros_like(y), 0
    for e in range(len(up)):
        t, j = torch.where(ids == e)  # in slot order, as the sorted rows are
        inner = y[t] @ up[e].t()
        inner = torch.relu(inner) if open_ is None else inner * open_[row:row + len(t)]
        row += len(t)
        out = out.index_add(0, t, (inner @ down[e].t()) * gate[t, j][:, None])
    return out, h


@pytest.mark.parametrize("shape", [(1, 2, 8, 512, 264), (65, 2, 8, 512, 264), (300, 6, 60, 264, 136)], ids=str)
def test_layer(gpu, shape):
    args = layer_inputs(*shape, seed=21)
    out, h = layer(*args)
    want, wh = layer_in_float64(gpu, args[0].cpu(), *(t.cpu().double() for t in args[1:]))
    # every step rounds once to binary16 (2^-11); five of them between x and the output
    assert float((out.cpu().double() - want).norm() / want.norm().clamp_min(1e-30)) < 5 * 2.0 ** -11
    assert float((h.cpu().double() - wh).abs().max()) <= 2.0 ** -11 * float(wh.abs().max())


def training_step(torch, leaves, ids, dout):
    x, r, w, gate, up, down = leaves
    y, h = tg.RmsNormFunction.apply(x, w, r, 1e-6)
    plan = tg.expert_sort(ids, len(up))
    xs = tg.ExpertGatherFunction.apply(y, *plan)
    inner = torch.relu(tg.ExpertGemmFunction.apply(xs, up, plan.offsets))
    out = tg.ExpertCombineFunction.apply(tg.ExpertGemmFunction.apply(inner, down, plan.offsets), gate, *plan)
    return (out, *torch.autograd.grad((out, h), leaves, (dout, dout)), inner)


def test_layer_training_step(gpu):
    """All gradients of a layer against float64 autograd of its definition."""
    ids, *vals = layer_inputs(200, 3, 8, 264, 136, seed=22)
    dout = gpu.randn(200, 264, generator=gpu.Generator().manual_seed(1)).half()
    got = training_step(gpu, [t.clone().requires_grad_() for t in vals], ids, dout.cuda())
    leaves = [t.cpu().double().requires_grad_() for t in vals]
    out, h = layer_in_float64(gpu, ids.cpu(), *leaves, (got[-1].detach() > 0).cpu())
    want = (out, *gpu.autograd.grad((out, h), leaves, (dout.double(), dout.double())))
    for name, a, b in zip(("out", "x", "r", "w", "gate", "up", "down"), got, want):
        # up to ten roundings of 2^-11 on the way
        assert float((a.detach().cpu().double() - b.detach()).norm() / b.detach().norm()) < 10 * 2.0 ** -11, name
        assert bool(gpu.isfinite(a).all()), name


def test_layer_on_a_stream_and_in_a_graph(gpu):
    """The layer captured once, its inputs (routing included) replaced between replays; and on a side
    stream given as an object and as a handle."""
    shape = (130, 4, 16, 264, 136)
    static = layer_inputs(*shape, seed=30)
    want = layer(*static)
    side = gpu.cuda.Stream()
    side.wait_stream(gpu.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = layer(*static, stream=stream)
        side.synchronize()
        assert gpu.equal(got[0], want[0]) and gpu.equal(got[1], want[1])
    graph = gpu.cuda.CUDAGraph()
    with gpu.cuda.graph(graph):
        out = layer(*static)
    for seed in (31, 32, 33):
        fresh = layer_inputs(*shape, seed=seed)
        eager = layer(*fresh)
        for s, f in zip(static, fresh):
            s.copy_(f)
        graph.replay()
        gpu.cuda.synchronize()
        assert gpu.equal(out[0], eager[0]) and gpu.equal(out[1], eager[1]), seed


def test_training_step_on_a_side_stream(gpu):
    ids, *vals = layer_inputs(130, 2, 8, 264, 136, seed=45)
    dout = gpu.full((130, 264), 0.5, dtype=gpu.float16, device="cuda")
    plain = training_step(gpu, [t.clone().requires_grad_() for t in vals], ids, dout)
    side = gpu.cuda.Stream()
    side.wait_stream(gpu.cuda.current_stream())
    with gpu.cuda.stream(side):
        other = training_step(gpu, [t.clone().requires_grad_() for t in vals], ids, dout)
    side.synchronize()
    gpu.cuda.synchronize()
    assert all(gpu.equal(a, b) for a, b in zip(plain, other))


def test_training_step_in_a_graph(gpu):
    shape = (130, 2, 8, 264, 136)
    ids, *vals = layer_inputs(*shape, seed=40)
    dout = gpu.full((130, 264), 0.5, dtype=gpu.float16, device="cuda")
    static = [t.clone().requires_grad_() for t in vals]
    side = gpu.cuda.Stream()
    side.wait_stream(gpu.cuda.current_stream())
    with gpu.cuda.stream(side):
        training_step(gpu, [t.clone().requires_grad_() for t in vals], ids, dout)
    side.synchronize()
    graph = gpu.cuda.CUDAGraph()
    with gpu.cuda.graph(graph, stream=side):
        out = [t.detach() for t in training_step(gpu, static, ids, dout)]
    for seed in (41, 42, 43):
        new_ids, *fresh = layer_inputs(*shape, seed=seed)
        eager = [t.detach() for t in training_step(gpu, [t.clone().requires_grad_() for t in fresh], new_ids, dout)]
        with gpu.no_grad():
            ids.copy_(new_ids)
            for s, f in zip(static, fresh):
                s.copy_(f)
        graph.replay()
        gpu.cuda.synchronize()
        assert all(gpu.equal(a, b) for a, b in zip(out, eager)), seed


def test_large_sort_in_two_graphs(gpu):
    """Two captured sorts of many slots (a workspace each, from the graph's own memory), replayed one
    after another and on two streams at once."""
    rng = np.random.default_rng(50)
    ids = [some_ids(rng, 40000, 2, 64, 0.1, np.int32) for _ in range(2)]
    dev = [to_dev(i) for i in ids]
    tg.expert_sort(dev[0], 64)
    graphs, plans = [], []
    for d in dev:
        g = gpu.cuda.CUDAGraph()
        with gpu.cuda.graph(g):
            plans.append(tg.expert_sort(d, 64))
        graphs.append(g)
    streams = [gpu.cuda.Stream(), gpu.cuda.Stream()]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with gpu.cuda.stream(s):
                g.replay()
        gpu.cuda.synchronize()
        for p, i in zip(plans, ids):
            check_sort(p, i, 64)


def test_saved_tensor_hooks(gpu):
    """Offloading hooks give the same gradients; a hook that returns another tensor is refused before
    its address reaches the library."""
    ids, *vals = layer_inputs(60, 2, 8, 264, 136, seed=60)
    dout = gpu.full((60, 264), 0.5, dtype=gpu.float16, device="cuda")

    def grads(pack, unpack):
        with gpu.autograd.graph.saved_tensors_hooks(pack, unpack):
            return training_step(gpu, [t.clone().requires_grad_() for t in vals], ids, dout)

    plain = grads(lambda t: t, lambda t: t)
    moved = grads(lambda t: t.cpu(), lambda t: t.cuda())
    assert all(gpu.equal(a, b) for a, b in zip(plain, moved))
    plan = tg.expert_sort(ids, 8)
    for bad in (lambda t: t[:1], lambda t: t.double(), lambda t: t.cpu()):
        for call in (lambda: tg.ExpertGatherFunction.apply(vals[0].clone().requires_grad_(), *plan),
                     lambda: tg.ExpertCombineFunction.apply(gpu.ones((120, 8), dtype=gpu.float16, device="cuda", requires_grad=True),
                                                            vals[3], *plan),
                     lambda: tg.ExpertGemmFunction.apply(gpu.ones((120, 264), dtype=gpu.float16, device="cuda", requires_grad=True),
                                                         vals[4], plan.offsets)):
            with gpu.autograd.graph.saved_tensors_hooks(lambda t: t, bad):
                out = call()
            with pytest.raises(RuntimeError, match="saved-tensor hook"):
                out.sum().backward()
