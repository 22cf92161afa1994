"""The GEMM's int32 sums on their own: no output, every path that writes them."""
import pytest
import torch

from w8a8_int8_quantized_qk_b200 import qk

pytestmark = pytest.mark.gpu

SIZES = [
    # one SM a tile: whole tiles of 256 and 128 columns, K split over a cluster
    (9, 264, 528), (40, 1032, 272), (128, 4096, 512), (100, 20480, 256), (128, 4096, 14336), (17, 8, 4096),
    # CTA pairs: whole tiles, K split over a cluster and through the workspace, the last wave's tiles cut
    (129, 136, 80), (257, 520, 528), (300, 2304, 1024), (512, 4104, 272), (256, 512, 8192), (4096, 4096, 512),
    (2305, 4096, 1040), (700, 8, 528),
]


def operands(m, n, k):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    a = torch.randint(-127, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    return a, b, torch.ones(m, device="cuda"), torch.ones(n, device="cuda")


@pytest.mark.parametrize("m,n,k", SIZES)
def test_sums_alone(m, n, k):
    """Exact (|sum| < 2^53), and nothing beyond the last row is written."""
    a, b, sa, sw = operands(m, n, k)
    want = (a.double() @ b.double().T).to(torch.int32)
    for _ in range(3):
        buf = torch.full((m + 3, n), -7, dtype=torch.int32, device="cuda")
        out, c = qk.w8a8_gemm(a, b, sa, sw, want_out=False, c=buf[:m])
        assert out is None and torch.equal(c, want)
        assert bool((buf[m:] == -7).all())
    _, both = qk.w8a8_gemm(a, b, sa, sw, want_c=True)
    assert torch.equal(both, want)
    assert qk.device_status() == qk.QK_OK


@pytest.mark.parametrize("m,n,k", [(40, 1032, 272), (300, 2304, 1024), (2305, 4096, 528)])
def test_sums_alone_asymmetric(m, n, k):
    a, b, sa, sw = operands(m, n, k)
    zp = (torch.arange(m, device="cuda") % 255 - 128).to(torch.int32)
    wsum = qk.weight_row_sums(b)
    out, c = qk.w8a8_gemm_asym(a, zp, b, wsum, sa, sw, want_out=False, want_c=True)
    want = a.double() @ b.double().T - zp.double()[:, None] * b.double().sum(1)
    assert out is None and torch.equal(c, want.to(torch.int32))
