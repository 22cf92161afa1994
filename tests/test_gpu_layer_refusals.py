"""GPU tests: what the helpers of the layer operators refuse before anything is launched."""
import pytest
import torch

from gpu_util import need_gpu
from w8a8_int8_quantized_qk_b200 import qk

pytestmark = pytest.mark.gpu


def calls():
    need_gpu()
    a = torch.ones((4, 64), dtype=torch.int8, device="cuda")
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    b = torch.ones((64, 64), dtype=torch.int8, device="cuda")
    s4, s64 = torch.ones(4, device="cuda"), torch.ones(64, device="cuda")
    la = torch.ones((2, 8, 64), dtype=torch.bfloat16, device="cuda")
    lb = torch.ones((2, 64, 8), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    w13 = torch.ones((3, 96, 64), dtype=torch.int8, device="cuda")
    w2 = torch.ones((3, 64, 48), dtype=torch.int8, device="cuda")
    s13, s2 = torch.ones((3, 96), device="cuda"), torch.ones((3, 64), device="cuda")
    return {"adapters": lambda ws: qk.w8a8_lora_gemm(a, b, s4, s64, x, la, lb, ids, workspace=ws),
            "moe layer": lambda ws: qk.w8a8_moe_layer(a, s4, ids[:, None], s4[:, None], w13, s13, w2, s2, workspace=ws)}


@pytest.mark.parametrize("operator", ["adapters", "moe layer"])
def test_workspaces(operator):
    call = calls()[operator]
    wide = torch.empty((1 << 12, 1 << 13), dtype=torch.uint8, device="cuda")
    want = call(None)
    for ws in (wide[0, :1].expand(1 << 24), wide.view(-1)[::2], wide[:, :4096], wide.cpu()):
        with pytest.raises(ValueError):
            call(ws)
    for ws in (wide, wide[256:], wide.view(torch.int32)):
        assert torch.equal(call(ws), want)
