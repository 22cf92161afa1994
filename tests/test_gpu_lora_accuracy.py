"""GPU tests of the accuracy of the adapters' products in their binary32 operands, fp32 tokens and s.  Those
enter the bf16 matrix instruction as three bf16 terms, x = h + m + l.

With u = 2^-24: the split is exact for every finite value, and so is a term's product with a power of two.  An
instruction adds its products to the accumulator and truncates to 24 bits; h, rounded, may lie one binade above
x, so that the three terms' sum is off by less than 2^-22 of x.  Where a row has one token element, all ranks
powers of two and each output one rank, no other sum is rounded, lora_scale's product is (2^-24): two operands
stay within 2 * 2^-22 + 2^-24, below EXACT = 2.5 * 2^-22.  The tokens and scales taken have |l| >= 2^-19 of
themselves, three times that, so that a product without its third term fails, however long k is.

Sums of many products: s is a chain of at most 8 instructions with the leading terms (2u each), those of the
smaller terms (2^-8 of it, 2u in all), at most k / 256 chains added (u each), 8 warps and 8 parts of K (u each) and
lora_scale (u); d is rank / 16 instructions (2u each) and its smaller terms (2u); the output's addition is one
more u.  In all (42 + k / 256 + rank / 8) u of the sum of the products' magnitudes."""
import pytest

from test_gpu_lora_range import one_rank_each, operands
from w8a8_int8_quantized_qk_b200 import qk

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

U = 2.0 ** -24
EXACT = 2.5 * 2.0 ** -22

# both sides of the boundary between short and long batches, every rank class of the output kernels
SIZES = [(1, 264, 16, 8), (5, 1032, 4112, 16), (40, 520, 1040, 24), (64, 264, 272, 128), (3, 136, 8208, 64),
         (65, 264, 4112, 16), (200, 520, 272, 32), (130, 264, 1040, 64), (300, 136, 528, 128), (1100, 136, 80, 72)]


def long_mantissas(count, seed):
    """Values in +-[1, 2) whose third bf16 term is at least 2^-19 of them."""
    g = torch.Generator().manual_seed(seed)
    v = 1.0 + torch.rand(16 * count + 64, generator=g)
    r = v - v.bfloat16().float()
    r = r - r.bfloat16().float()
    assert torch.equal(r, r.bfloat16().float())  # (nothing is left)
    v = v[r.abs() >= v * 2.0 ** -19][:count]
    assert len(v) == count
    return v * (1.0 - 2.0 * torch.randint(0, 2, (count,), generator=g))


@pytest.mark.parametrize("m,n,k,rank", SIZES)
@pytest.mark.parametrize("x_dtype", [torch.float32, torch.bfloat16])
def test_three_terms(m, n, k, rank, x_dtype):
    adapters = 3
    values = long_mantissas(m + adapters, m + k)
    lora_a = (2.0 ** -(torch.arange(rank) % 3).float())[None, :, None].expand(adapters, rank, k)
    lora_b = one_rank_each(n, rank, adapters)
    x = torch.zeros((m, k))
    at = torch.arange(m) * 37 % k
    if x_dtype == torch.float32:
        x[torch.arange(m), at] = values[:m]  # 24 bits in the token, and so in s
        scale = None
    else:
        x[torch.arange(m), at] = 2.0 ** (torch.arange(m) % 5).float()
        scale = values[m:]                   # 24 bits in s alone
    p = operands(m, n, k, rank, adapters, x.to(x_dtype), lora_a, lora_b, scale)
    got = qk.w8a8_lora_gemm(**p, out_dtype=torch.float32).double().cpu()
    ids = p["adapter_ids"].cpu().long()
    s = x.double().sum(1)[:, None] * lora_a[0, :, 0].double()[None]
    if scale is not None:
        s = s * scale.double()[ids][:, None]
    want = torch.einsum("ir,ijr->ij", s, lora_b.double()[ids])
    assert bool((want != 0).all())
    assert float(((got - want) / want).abs().max()) <= EXACT
    assert qk.device_status() == qk.QK_OK


@pytest.mark.parametrize("m,n,k,rank", SIZES)
@pytest.mark.parametrize("x_dtype", [torch.float32, torch.bfloat16])
def test_sums_of_many_products(m, n, k, rank, x_dtype):
    adapters = 3
    g = torch.Generator().manual_seed(m + n + k)
    x = torch.randn((m, k), generator=g).to(x_dtype)
    p = operands(m, n, k, rank, adapters, x, torch.randn((adapters, rank, k), generator=g) / k ** 0.5,
                 torch.randn((adapters, n, rank), generator=g) / rank ** 0.5, 0.25 + torch.rand(adapters, generator=g))
    got = qk.w8a8_lora_gemm(**p, out_dtype=torch.float32).double()
    ids = p["adapter_ids"].long()
    for e in range(adapters):
        rows = (ids == e).nonzero()[:, 0]
        la, lb, ls = p["lora_a"][e].double(), p["lora_b"][e].double(), p["lora_scale"][e].double()
        xs = p["x"][rows].double()
        want, mag = ls * ((xs @ la.T) @ lb.T), ls * ((xs.abs() @ la.abs().T) @ lb.abs().T)
        assert bool(((got[rows] - want).abs() <= (42 + k / 256 + rank / 8) * U * mag).all())
