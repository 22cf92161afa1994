"""GPU tests of the layer operators where offsets pass 32 bits: the last rows of a long batch, and the last of many
experts, agree bit for bit with the same rows, or expert, on their own."""
import pytest

from gpu_util import need_gpu
from w8a8_int8_quantized_qk_b200 import qk

pytestmark = pytest.mark.gpu

import torch  # noqa: E402


@pytest.fixture(autouse=True)
def room():
    need_gpu()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    yield
    torch.cuda.empty_cache()


def rand8(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)


@pytest.mark.parametrize("m,k", [(270000, 8192), (66000, 32784)])
def test_norm(m, k):
    """A walked form and a cluster's (fewer rows may take another one: the same codes, which depend on no sum; each
    scale within (k / 256 + 16) / 2 + 8 steps of 2^-24 of the exact one, and each normalised value half a bf16 step
    more, so that two are twice that apart)."""
    assert m * k > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((m, k), dtype=torch.bfloat16, device="cuda")
    x[:1000].normal_(generator=g)
    x[-1000:].normal_(generator=g)
    x[1000:-1000] = 1.0
    w = (1 + 0.1 * torch.randn(k, generator=g, device="cuda")).bfloat16()
    last = x[-5:].clone()
    q, s, r, y = qk.add_rmsnorm_quant_per_token(x, w, x, want_norm=True, residual_out=x)  # x + x in place
    q1, s1, r1, y1 = qk.add_rmsnorm_quant_per_token(last, w, last.clone(), want_norm=True)
    assert torch.equal(q[-5:], q1) and torch.equal(r[-5:], r1)
    tol = ((k / 256 + 16) / 2 + 8) * 2.0 ** -24
    assert bool(((s[-5:] - s1).abs() <= 2 * tol * s1).all())
    assert bool(((y[-5:].float() - y1.float()).abs() <= (2.0 ** -7 + 2 * tol) * y1.float().abs()).all())


def test_adapters():
    m, n, k, rank = 147000, 14720, 64, 8
    assert m * n > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(2)
    a, b = rand8(g, m, k), rand8(g, n, k)
    sa, sw = torch.rand(m, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda") / 1000
    x = torch.randn((m, k), generator=g, device="cuda").bfloat16()
    la = torch.randn((3, rank, k), generator=g, device="cuda").bfloat16()
    lb = torch.randn((3, n, rank), generator=g, device="cuda").bfloat16()
    ids = torch.randint(-1, 3, (m,), generator=g, device="cuda", dtype=torch.int32)
    out = qk.w8a8_lora_gemm(a, b, sa, sw, x, la, lb, ids)
    plain, _ = qk.w8a8_gemm(a[-300:], b, sa[-300:], sw)
    rows = (ids[-300:] < 0).nonzero()[:, 0]
    assert torch.equal(out[-300:][rows], plain[rows])
    want = plain.double()
    for e in range(3):
        use = (ids[-300:] == e).nonzero()[:, 0]
        want[use] = ((a[-300:][use].double() @ b.double().T) * sa[-300:][use].double()[:, None] * sw.double()
                     + (x[-300:][use].double() @ la[e].double().T) @ lb[e].double().T)
    # half a bf16 step of the result (of the reference's own, too, for rows without an adapter); the sums within
    # 44 * 2^-24 of the products' magnitudes together, which stay below 2^11 (8 ranks of 64 products)
    assert bool(((out[-300:].double() - want).abs() <= want.abs() * 2.0 ** -7 + 2.0 ** -7).all())


def test_adapters_of_large_stacks():
    """The last adapter's rows lie behind 2^32 bytes of lora_a and of lora_b."""
    m, n, k, rank, adapters = 70, 2048, 2048, 128, 8200
    assert adapters * rank * k * 2 > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(3)
    la = torch.zeros((adapters, rank, k), dtype=torch.bfloat16, device="cuda")
    lb = torch.zeros((adapters, n, rank), dtype=torch.bfloat16, device="cuda")
    la[-2:].normal_(generator=g)
    lb[-2:].normal_(generator=g)
    b, sw = rand8(g, n, k), torch.rand(n, generator=g, device="cuda") / 1000
    for rows in (m, 9):
        x = torch.randn((rows, k), generator=g, device="cuda").bfloat16()
        a, sa = qk.quantize_per_token(x)
        ids = (torch.arange(rows, device="cuda") % 2).to(torch.int32)
        far = qk.w8a8_lora_gemm(a, b, sa, sw, x, la, lb, ids + adapters - 2)
        near = qk.w8a8_lora_gemm(a, b, sa, sw, x, la[-2:].clone(), lb[-2:].clone(), ids)
        assert torch.equal(far, near)


def test_moe_layer():
    """The last expert's rows lie behind 2^32 bytes of w_gate_up and 2^31 of w_down."""
    m, experts, hidden, inter = 5, 130, 2048, 8192
    assert experts * 2 * inter * hidden > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(4)
    w13 = torch.zeros((experts, 2 * inter, hidden), dtype=torch.int8, device="cuda")
    w2 = torch.zeros((experts, hidden, inter), dtype=torch.int8, device="cuda")
    w13[-2:], w2[-2:] = rand8(g, 2, 2 * inter, hidden), rand8(g, 2, hidden, inter)
    s13 = torch.rand((experts, 2 * inter), generator=g, device="cuda") / 5000
    s2 = torch.rand((experts, hidden), generator=g, device="cuda") / 5000
    a, sa = rand8(g, m, hidden), torch.rand(m, generator=g, device="cuda") / 100
    top = torch.tensor([[0, 1], [1, 0], [1, -3], [-3, -3], [0, 0]], dtype=torch.int32, device="cuda")
    wt = torch.rand((m, 2), generator=g, device="cuda")
    far = qk.w8a8_moe_layer(a, sa, torch.where(top < 0, top, top + experts - 2), wt, w13, s13, w2, s2)
    near = qk.w8a8_moe_layer(a, sa, top, wt, w13[-2:].clone(), s13[-2:].clone(), w2[-2:].clone(), s2[-2:].clone())
    assert bool(near[:3].float().abs().max() > 0) and torch.equal(far, near)
