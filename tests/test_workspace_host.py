"""Host-side tests (nothing is launched): a caller's workspace is taken for as many bytes as it has elements,
from its first one on, so it has to be dense.  An expanded tensor has fewer bytes than elements, and the gaps
of a strided view belong to somebody else."""
import pytest

from w8a8_int8_quantized_qk_b200 import qk

torch = pytest.importorskip("torch")


class OnDevice(torch.Tensor):
    """A host tensor that says it lies on device 0."""

    is_cuda = True

    def get_device(self):
        return 0


def on_device(t):
    return t.as_subclass(OnDevice)


def strided():
    return [torch.empty(1, dtype=torch.uint8).expand(1 << 20),      # one byte of storage
            torch.empty(2 << 20, dtype=torch.uint8)[::2],           # every second byte
            torch.empty(1024, 2048, dtype=torch.uint8)[:, :1024],   # a block of columns
            torch.empty(1, 1024, dtype=torch.int32).expand(256, 1024)]


@pytest.mark.parametrize("at", range(4))
def test_operator_workspaces_are_dense(at):
    with pytest.raises(ValueError, match="workspace: must be contiguous"):
        qk._workspace(on_device(strided()[at]), 4096, 0, "cpu")


def test_operator_workspaces_taken():
    for ws in (torch.empty(4096, dtype=torch.uint8), torch.empty(8192, dtype=torch.uint8)[1024:],
               torch.empty(64, 64, dtype=torch.int32), torch.empty(4, 1024, dtype=torch.uint8)[1:2]):
        address, size, hold = qk._workspace(on_device(ws), 4096, 0, "cpu")
        assert (address, size) == (ws.data_ptr(), ws.numel() * ws.element_size()) and hold is not None
    assert qk._workspace(None, 0, 0, "cpu") == (None, 0, None)
    with pytest.raises(ValueError, match="on device 0, others on 1"):
        qk._workspace(on_device(torch.empty(4096, dtype=torch.uint8)), 4096, 1, "cpu")


@pytest.mark.parametrize("at", range(4))
@pytest.mark.parametrize("helper", ["w8a8_gemm", "w8a8_gemm_asym", "w8a8_linear", "w8a8_linear_fused"])
def test_gemm_workspaces_are_dense(helper, at):
    ws = on_device(strided()[at])
    a, b = (on_device(torch.zeros(s, dtype=torch.int8)) for s in ((4, 64), (16, 64)))
    x = on_device(torch.zeros((4, 64), dtype=torch.bfloat16))
    sa, sw = (on_device(torch.ones(s)) for s in (4, 16))
    zp, wsum = (on_device(torch.zeros(s, dtype=torch.int32)) for s in (4, 16))
    call = {"w8a8_gemm": lambda: qk.w8a8_gemm(a, b, sa, sw, workspace=ws),
            "w8a8_gemm_asym": lambda: qk.w8a8_gemm_asym(a, zp, b, wsum, sa, sw, workspace=ws),
            "w8a8_linear": lambda: qk.w8a8_linear(x, b, sw, workspace=ws),
            "w8a8_linear_fused": lambda: qk.w8a8_linear_fused(x, b, sw, workspace=ws)}[helper]
    with pytest.raises(ValueError, match="workspace: must be contiguous"):
        call()
