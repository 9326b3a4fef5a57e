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
