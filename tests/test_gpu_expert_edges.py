"""The expert layer's operators at the ends of what they accept."""
import numpy as np
import pytest

import expert_reference as ref
from gpu_util import to_dev, torch_cuda
from test_gpu_experts import ROWS_ONLY, exact_product, groups, small_ints

import tiled_dense_gemm_04_amd as tg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = torch_cuda()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tg.lib()
    return torch


@pytest.mark.parametrize("H", [1, 7, 64, 4100])
def test_gather_without_choices(gpu, H):
    """Tokens without slots, through the C entry point: the rows behind offsets[E] are zeroed, the others
    left as they were, and neither x nor place is needed."""
    rows, used = 100, 37
    out = gpu.full((rows, H), 3.0, dtype=gpu.float16, device="cuda")
    offsets = to_dev(np.array([0, 5, used], dtype=np.int32))
    stream = gpu.cuda.current_stream().cuda_stream
    for tokens in (0, 1, 700):
        out.fill_(3.0)
        assert tg.lib().expert_gather_f16(tokens, 0, rows, H, None, H, None, out.data_ptr(), H, offsets.data_ptr(), 2,
                                          stream) == tg.TGEMM_OK
        assert (out[:used] == 3).all() and (out[used:] == 0).all()


def test_zeroed_rows_near_the_largest_index(gpu):
    """As many rows as the entry points take: those behind the last in use are zeroed, and no others."""
    rows = (1 << 31) - 1
    used = rows - 1000
    out = gpu.full((rows,), 3.0, dtype=gpu.float16, device="cuda")  # 4.3 GB
    offsets = to_dev(np.array([0, 9, used], dtype=np.int32))
    stream = gpu.cuda.current_stream().cuda_stream
    L = tg.lib()
    assert L.expert_gather_f16(0, 0, rows, 1, None, 1, None, out.data_ptr(), 1, offsets.data_ptr(), 2, stream) == tg.TGEMM_OK
    assert (out[used:] == 0).all() and (out[used - 1000:used] == 3).all() and (out[:4096] == 3).all()
    out[used:] = 3.0
    assert L.expert_combine_f16_backward(0, 0, rows, 1, None, 1, None, 1, None, None, 1, out.data_ptr(), 1, None,
                                         offsets.data_ptr(), 2, stream) == tg.TGEMM_OK
    assert (out[used:] == 0).all() and (out[used - 1000:used] == 3).all() and (out[:4096] == 3).all()


def saved_by(gpu, call):
    """(outputs of call, the shapes of what its functions keep for their backward passes)."""
    shapes = []

    def pack(t):
        shapes.append(tuple(t.shape))
        return t

    with gpu.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        return call(), sorted(shapes)


def test_combine_keeps_its_rows_for_the_weights_gradient_only(gpu):
    """The rows (T k x H) are held, and may not be changed in place, only where a weight's gradient reads them."""
    rng = np.random.default_rng(1)
    T, k, E, H = 40, 3, 8, 264
    plan = tg.expert_sort(to_dev(rng.integers(0, E, (T, k))), E)
    y, w = to_dev(rng.standard_normal((T * k, H)).astype(np.float16)), to_dev(rng.random((T, k)).astype(np.float32))
    dout = to_dev(rng.standard_normal((T, H)).astype(np.float16))
    full = [y.clone().requires_grad_(), w.clone().requires_grad_()]
    out, kept = saved_by(gpu, lambda: tg.ExpertCombineFunction.apply(*full, *plan))
    assert (T * k, H) in kept
    dy, dw = gpu.autograd.grad(out, full, dout, retain_graph=True)
    for leaf, want in zip(full, (dy, dw)):  # more kept than the one gradient reads
        assert gpu.equal(gpu.autograd.grad(out, leaf, dout, retain_graph=True)[0], want)
    rows = y.clone().requires_grad_()
    inner = rows * 1
    out, kept = saved_by(gpu, lambda: tg.ExpertCombineFunction.apply(inner, w, *plan))
    assert kept == sorted([(E + 1,), (T, k), (T, k)])
    inner.detach().zero_()  # what the backward pass does not read may change
    assert gpu.equal(gpu.autograd.grad(out, rows, dout)[0], dy)
    out, kept = saved_by(gpu, lambda: tg.ExpertCombineFunction.apply(rows, None, *plan))
    assert kept == sorted([(E + 1,), (T, k)])
    gate = w.clone().requires_grad_()
    out, kept = saved_by(gpu, lambda: tg.ExpertCombineFunction.apply(y, gate, *plan))
    assert (T * k, H) in kept and gpu.equal(gpu.autograd.grad(out, gate, dout)[0], dw)


def test_products_keep_an_operand_for_the_others_gradient_only(gpu):
    """Frozen experts need no rows kept, and rows without a gradient no experts."""
    rng = np.random.default_rng(2)
    rows, E, N, K = 50, 3, 40, 64
    a, b, dc = (to_dev(rng.integers(-2, 3, s).astype(np.float16)) for s in ((rows, K), (E, N, K), (rows, N)))
    offsets = to_dev(np.array([0, 20, 20, 47], dtype=np.int32))
    both = [a.clone().requires_grad_(), b.clone().requires_grad_()]
    out, kept = saved_by(gpu, lambda: tg.ExpertGemmFunction.apply(*both, offsets))
    assert kept == sorted([(E + 1,), (rows, K), (E, N, K)])
    da, db = gpu.autograd.grad(out, both, dc, retain_graph=True)
    for leaf, want in zip(both, (da, db)):
        assert gpu.equal(gpu.autograd.grad(out, leaf, dc, retain_graph=True)[0], want)
    out, kept = saved_by(gpu, lambda: tg.ExpertGemmFunction.apply(both[0], b, offsets))
    assert kept == sorted([(E + 1,), (E, N, K)])
    assert gpu.equal(gpu.autograd.grad(out, both[0], dc)[0], da)
    inner = a.clone()
    out, kept = saved_by(gpu, lambda: tg.ExpertGemmFunction.apply(inner, both[1], offsets))
    assert kept == sorted([(E + 1,), (rows, K)])
    assert gpu.equal(gpu.autograd.grad(out, both[1], dc)[0], db)
    # both operands strided where the hooks give them back
    with gpu.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: t.repeat_interleave(2, dim=-1)[..., ::2]):
        out = tg.ExpertGemmFunction.apply(*both, offsets)
    assert all(gpu.equal(g, w) for g, w in zip(gpu.autograd.grad(out, both, dc), (da, db)))


def uneven(E, seed):
    """Counts of E experts, a few with most of the rows, some with none."""
    rng = np.random.default_rng(seed)
    counts = rng.integers(0, 40, E)
    counts[rng.integers(0, E, max(1, E // 8))] = rng.integers(300, 900, max(1, E // 8))
    return counts


@pytest.mark.parametrize("cfg", [None, tg.EXPERT_GENERIC, tg.EXPERT_128, tg.EXPERT_256, tg.EXPERT_TILES], ids=lambda c: f"cfg{c}")
@pytest.mark.parametrize("E", [7, 8, 33, 63, 64, 65, 130])
def test_weights_form_of_many_experts(gpu, E, cfg):
    """Experts ranked by their rows, one a lane, up to 64 of them, and more than that: equal ones, one that
    has all rows, and uneven ones, where there are big tiles, quarters and edges."""
    rng = np.random.default_rng(E)
    one = np.zeros(E, dtype=np.int64)
    one[E // 2] = 700
    for name, counts in (("equal", np.full(E, 33)), ("one", one), ("uneven", uneven(E, 1)), ("longest first", -np.sort(-uneven(E, 2))),
                         ("longest last", np.sort(uneven(E, 3)))):
        offsets, rows = groups(counts, 3)
        for N, M in ((520, 1000), (264, 136)) if name == "uneven" else ((520, 1000),) if E < 100 else ((264, 392),):
            print(f"E {E} cfg {cfg} {name} {rows} rows {M} x {N}", flush=True)
            got, want = exact_product("tn", rng, offsets, rows, N, M, cfg)
            assert np.array_equal(got, want), (name, M, N)


def padded(gpu, x, ld, value=float("nan")):
    """x in rows of ld elements, all around it `value`."""
    rows, cols = x.shape
    buf = gpu.full((rows + 2, ld), value, dtype=gpu.float16, device="cuda")
    view = buf[1:rows + 1, :cols]
    view.copy_(to_dev(x))
    return view


EVERY = [None, tg.EXPERT_GENERIC, tg.EXPERT_32, tg.EXPERT_64, tg.EXPERT_128, tg.EXPERT_256, tg.EXPERT_TILES]


@pytest.mark.parametrize("poison", [False, True], ids=["product", "poisoned"])
@pytest.mark.parametrize("cfg", EVERY, ids=lambda c: f"cfg{c}")
@pytest.mark.parametrize("form", ["nt", "nn"])
def test_nothing_past_an_operands_end_is_multiplied(gpu, form, cfg, poison):
    """NaN behind every row's end, before the first row and behind the last, and in the rows of no expert:
    one that either operand let in would show, as the other's zeros do not hide it."""
    library = tg.debugfill_lib() if poison else None
    rng = np.random.default_rng(7)
    counts = [33, 0, 129, 300, 1]
    offsets, rows = groups(counts, 6)
    E = len(counts)
    for N, K in ((8, 8), (40, 64), (136, 72), (264, 200), (520, 40)) + (((37, 61), (130, 3)) if cfg in (None, tg.EXPERT_GENERIC) else ()):
        a = small_ints(rng, rows, K).astype(np.float64)
        b = small_ints(rng, E, N, K) if form == "nt" else small_ints(rng, E, K, N)
        want, _ = ref.products(a, b, offsets, form == "nt", np.full((rows, N), 7.0))
        a[offsets[-1]:] = np.nan
        pad = 8 if K % 8 == 0 and N % 8 == 0 else 3
        r, c = b.shape[1:]
        buf = gpu.full((E, r + 2, c + pad), float("nan"), dtype=gpu.float16, device="cuda")
        bv = buf[:, 1:r + 1, :c]
        bv.copy_(to_dev(b))
        out = gpu.full((rows, N), 7.0, dtype=gpu.float16, device="cuda")
        tg.expert_gemm_f16(padded(gpu, a.astype(np.float16), K + pad), bv, to_dev(offsets), out, trans_b=form == "nt", cfg=cfg,
                           library=library)
        assert np.array_equal(out.cpu().numpy(), ref.to_half(want)), (N, K)


@pytest.mark.parametrize("poison", [False, True], ids=["product", "poisoned"])
@pytest.mark.parametrize("cfg", [c for c in EVERY if c not in ROWS_ONLY], ids=lambda c: f"cfg{c}")
def test_a_nan_stays_in_its_expert_of_the_weights_form(gpu, cfg, poison):
    """Every other expert's rows NaN in one operand or both, and all around the operands: the experts between
    are exact, and the others' results NaN."""
    library = tg.debugfill_lib() if poison else None
    rng = np.random.default_rng(8)
    counts = [5, 33, 0, 64, 7, 129, 300, 20, 63, 31]
    offsets, rows = groups(counts, 6)
    E = len(counts)
    for M, N in ((8, 8), (40, 264), (136, 520), (392, 72)) + (((37, 61),) if cfg in (None, tg.EXPERT_GENERIC) else ()):
        a, b = small_ints(rng, rows, M), small_ints(rng, rows, N)
        want = ref.to_half(ref.products_tn(a, b, offsets))
        pad = 8 if M % 8 == 0 and N % 8 == 0 else 3
        for dirty in ("a", "b", "both"):
            av, bv = padded(gpu, a, M + pad), padded(gpu, b, N + pad)
            for e in range(0, E, 2):
                lo, hi = int(offsets[e]), int(offsets[e + 1])
                if dirty != "b":
                    av[lo:hi] = float("nan")
                if dirty != "a":
                    bv[lo:hi] = float("nan")
            av[int(offsets[-1]):], bv[int(offsets[-1]):] = float("nan"), float("nan")
            got = tg.expert_gemm_f16_tn(av, bv, to_dev(offsets), cfg=cfg, library=library).cpu().numpy()
            assert np.array_equal(got[1::2], want[1::2]), (M, N, dirty)
            for e in range(0, E, 2):
                assert np.isnan(got[e]).all() if counts[e] else (got[e] == 0).all()
