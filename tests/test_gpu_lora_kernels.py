"""GPU tests of which kernels an adapters' call launches."""
import pytest

from gpu_util import need_gpu
from w8a8_int8_quantized_qk_b200 import qk

pytestmark = pytest.mark.gpu

import torch  # noqa: E402


def kernels(m, rank, x_dtype):
    n, k = 136, 272
    a = torch.ones((m, k), dtype=torch.int8, device="cuda")
    b = torch.ones((n, k), dtype=torch.int8, device="cuda")
    la = torch.ones((2, rank, k), dtype=torch.bfloat16, device="cuda")
    lb = torch.ones((2, n, rank), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(m, dtype=torch.int32, device="cuda")
    sa, sw, x = torch.ones(m, device="cuda"), torch.ones(n, device="cuda"), torch.ones((m, k), device="cuda").to(x_dtype)
    qk.w8a8_lora_gemm(a, b, sa, sw, x, la, lb, ids)
    torch.cuda.synchronize()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
        qk.w8a8_lora_gemm(a, b, sa, sw, x, la, lb, ids)
        torch.cuda.synchronize()
    return {e.name for e in p.events() if "lora" in e.name}


@pytest.mark.parametrize("rank", [8, 16, 24, 64, 128])
@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
def test_short_and_long_batches_share_no_kernel(rank, x_dtype):
    """A short batch's kernels ask for a split of L1 and shared memory that stays with them: none of a long batch's may
    be among them, or a call would run slower for another one before it."""
    need_gpu()
    short, long_ = kernels(64, rank, x_dtype), kernels(65, rank, x_dtype)
    if not short or not long_:
        pytest.skip("no kernel names from the profiler")
    assert any("shrink" in name for name in short) and any("shrink" in name for name in long_)
    assert not short & long_
