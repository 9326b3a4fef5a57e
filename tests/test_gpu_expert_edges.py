"""The expert layer's operators at the ends of what they accept."""
import numpy as np
import pytest

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
