"""The MXFP4 autograd forms under saved-tensor hooks (checkpointing, offloading, copies): output
and gradients bit for bit those without hooks."""
import gc

import numpy as np
import pytest

from gpu_util import log, torch_cuda

import tiled_dense_gemm_04_amd as tg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = torch_cuda()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tg.lib()
    return torch


def contexts(torch):
    from torch.autograd.graph import save_on_cpu, saved_tensors_hooks
    from torch.utils.checkpoint import checkpoint

    def under(ctx):
        def run(fn, *args):
            with ctx():
                return fn(*args)
        return run

    return {"checkpoint": lambda fn, *args: checkpoint(fn, *args, use_reentrant=False),
            "reentrant checkpoint": lambda fn, *args: checkpoint(fn, *args, use_reentrant=True),
            "on the CPU": under(save_on_cpu),
            "copies": under(lambda: saved_tensors_hooks(lambda t: t.clone(), lambda t: t.clone()))}


# The kept block (4-bit X^T and W^T) is far larger than a gradient, or of a gradient's size class.
@pytest.mark.parametrize("M,N,K", [(200, 200, 200), (100, 264, 200), (33, 40, 1000), (2048, 512, 512), (16384, 4096, 4096)])
@pytest.mark.parametrize("form", ["linear", "weight"])
def test_gradients_under_hooks(gpu, form, M, N, K):
    gen = gpu.Generator(device="cuda").manual_seed(M + N + K)

    def normal(*shape):
        return gpu.randn(*shape, generator=gen, device="cuda").half()

    x, w, dy = normal(M, K), normal(N, K) / 16, normal(M, N)
    codes = tg.mxfp4_quant(w)
    leaves = [x.requires_grad_()] + ([w.requires_grad_()] if form == "linear" else [])

    def layer(*args):
        if form == "linear":
            return tg.Mxfp4LinearFunction.apply(*args)
        return tg.Mxfp4WeightFunction.apply(*args, *codes)

    def step(run):
        for t in leaves:
            t.grad = None
        y = run(layer, *leaves)
        y.backward(dy)
        gpu.cuda.synchronize()
        return [y.detach().cpu().numpy()] + [t.grad.cpu().numpy() for t in leaves]

    want = step(lambda fn, *args: fn(*args))
    for name, run in contexts(gpu).items():
        log(f"{form} {M}x{N}x{K}: {name}")
        # no cached free blocks: memory given back too early is what the next allocation gets
        gc.collect()
        gpu.cuda.empty_cache()
        for got, ref in zip(step(run), want):
            assert np.array_equal(got, ref), name


def test_two_layers_in_one_checkpoint(gpu):
    """A checkpointed pair of layers: the backward of the second runs while the first's block waits."""
    from torch.utils.checkpoint import checkpoint
    gen = gpu.Generator(device="cuda").manual_seed(7)
    x, w1, w2 = (gpu.randn(*s, generator=gen, device="cuda").half().requires_grad_() for s in ((300, 256), (512, 256), (256, 512)))
    dy = gpu.randn(300, 256, generator=gen, device="cuda").half()

    def block(a, u, v):
        return tg.Mxfp4LinearFunction.apply(gpu.relu(tg.Mxfp4LinearFunction.apply(a, u) * 0.0625), v)

    want = gpu.autograd.grad(block(x, w1, w2), (x, w1, w2), dy)
    got = gpu.autograd.grad(checkpoint(block, x, w1, w2, use_reentrant=False), (x, w1, w2), dy)
    for a, b in zip(got, want):
        assert gpu.equal(a, b)
