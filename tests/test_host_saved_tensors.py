"""Mxfp4LinearFunction's backward under saved-tensor hooks, on the CPU: the library's calls are
replaced by ones that look at the memory they are handed (an unpacked tensor may have no other
owner than the backward pass itself)."""
import weakref

import pytest
import torch

from tiled_dense_gemm_04_amd import mxfp4


@pytest.fixture
def calls(monkeypatch):
    """The products' calls: (operand B's address, the saved storages alive then)."""
    seen, unpacked = [], []

    def alive():
        return [(s.data_ptr(), s.data_ptr() + s.nbytes()) for s in (r() for r in unpacked) if s is not None]

    def packed_gemm(a, a_base, b, b_base, device):
        seen.append((b_base + b[2], b[0] * (b[3] + b[5]), alive()))
        return torch.zeros((a[0], b[0]), dtype=torch.float16)

    monkeypatch.setattr(mxfp4, "_row_major", lambda x, name: x)
    monkeypatch.setattr(mxfp4, "_packed_quant", lambda *args: None)
    monkeypatch.setattr(mxfp4, "_packed_gemm", packed_gemm)
    return seen, unpacked


def linear(x, w):
    return mxfp4.autograd_functions()["Mxfp4LinearFunction"].apply(x, w)


@pytest.mark.parametrize("grads", [(True, True), (True, False), (False, True)])
def test_unpacked_copy_lives_until_both_products(calls, grads):
    seen, unpacked = calls

    def unpack(t):
        t = t.clone()
        unpacked.append(weakref.ref(t.untyped_storage()))
        return t

    x = torch.ones(70, 100, dtype=torch.float16, requires_grad=grads[0])
    w = torch.ones(40, 100, dtype=torch.float16, requires_grad=grads[1])
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
        y = linear(x, w)
    seen.clear()
    y.backward(torch.ones_like(y))
    assert len(seen) == sum(grads)
    for begin, nbytes, alive in seen:
        assert any(lo <= begin and begin + nbytes <= hi for lo, hi in alive), \
            "the product reads a saved operand whose memory has been given back"


def test_kept_block_lives_in_a_checkpoint(calls):
    """A non-reentrant checkpoint hands the backward pass tensors of a second forward pass."""
    from torch.utils.checkpoint import checkpoint
    seen, unpacked = calls
    save = torch.autograd.function.FunctionCtx.save_for_backward

    def save_for_backward(ctx, *tensors):
        unpacked.extend(weakref.ref(t.untyped_storage()) for t in tensors)
        return save(ctx, *tensors)

    fn = mxfp4.autograd_functions()["Mxfp4LinearFunction"]
    x = torch.ones(70, 100, dtype=torch.float16, requires_grad=True)
    w = torch.ones(40, 100, dtype=torch.float16, requires_grad=True)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(torch.autograd.function.FunctionCtx, "save_for_backward", save_for_backward)
        y = checkpoint(fn.apply, x, w, use_reentrant=False)
        seen.clear()
        y.backward(torch.ones_like(y))
    products = seen[1:]  # the second forward pass, then dx and dw
    assert len(products) == 2
    for begin, nbytes, alive in products:
        assert any(lo <= begin and begin + nbytes <= hi for lo, hi in alive)


@pytest.mark.parametrize("wrong", [lambda t: t[:-1], lambda t: t.to("meta"), lambda t: t.float(), lambda t: t.repeat_interleave(2)[::2]],
                         ids=["shorter", "elsewhere", "another type", "strided"])
def test_a_hook_that_returns_something_else_is_refused(calls, wrong):
    """The products take addresses: a saved block that is not the forward pass's must not reach them."""
    seen, _ = calls
    x = torch.ones(70, 100, dtype=torch.float16, requires_grad=True)
    w = torch.ones(40, 100, dtype=torch.float16, requires_grad=True)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, wrong):
        y = linear(x, w)
    seen.clear()
    with pytest.raises(RuntimeError, match="saved"):
        y.backward(torch.ones_like(y))
    assert not seen
