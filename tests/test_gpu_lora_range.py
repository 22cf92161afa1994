"""GPU tests of the adapters' operands at the ends of the range: binary32 tokens and s up to the largest value
(which lies above the largest of bf16, whose terms they are taken apart into), and infinite ones.

A power of two times a value of one token element, one rank an output and no other product: the three terms add
up to it; an instruction truncates to 24 bits and the first term, rounded, may lie one binade above the value, so
each of the two products is off by less than 2^-22 of it, 2.5 * 2^-22 in all with lora_scale's rounding."""
import numpy as np
import pytest

from gpu_util import need_gpu
from w8a8_int8_quantized_qk_b200 import qk

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

EXACT = 2.5 * 2.0 ** -22
BIG = float(np.finfo(np.float32).max)


def operands(m, n, k, rank, adapters, x, lora_a, lora_b, lora_scale=None, ids=None):
    """A projection whose own part is zero."""
    need_gpu()
    a = torch.ones((m, k), dtype=torch.int8, device="cuda")
    b = torch.ones((n, k), dtype=torch.int8, device="cuda")
    if ids is None:
        ids = (torch.arange(m) % adapters).to(torch.int32)
    return dict(a=a, b=b, scale_a=torch.ones(m, device="cuda"), scale_b=torch.zeros(n, device="cuda"), x=x.cuda(),
                lora_a=lora_a.bfloat16().cuda(), lora_b=lora_b.bfloat16().cuda(), adapter_ids=ids.cuda(),
                lora_scale=None if lora_scale is None else lora_scale.cuda())


def one_rank_each(n, rank, adapters):
    """lora_b with one power of two in each output's row, and where it stands."""
    j, e = torch.arange(n), torch.arange(adapters)
    at = (j[None] * 7 + e[:, None]) % rank
    b = torch.zeros((adapters, n, rank))
    b.scatter_(2, at[..., None], (2.0 ** (j % 4).float()).expand(adapters, n)[..., None])
    return b


@pytest.mark.parametrize("m,n,k,rank", [(1, 264, 16, 8), (20, 136, 528, 16), (64, 136, 272, 128), (66, 136, 528, 16),
                                        (130, 136, 80, 32), (200, 136, 272, 64), (80, 136, 272, 128)])
@pytest.mark.parametrize("where", ["token", "s"])
def test_largest_finite_values(m, n, k, rank, where):
    """Up to the largest binary32 value, which lies above the largest of bf16."""
    adapters = 2
    big = torch.tensor([BIG, -BIG, 3.3953e38, 3.3954e38, -3.4e38, 1.0])[torch.arange(m) % 6]
    x = torch.zeros((m, k))
    x[torch.arange(m), torch.arange(m) * 5 % k] = big
    # s is x's own size, or 2^-40 of it
    lora_a = torch.full((adapters, rank, k), 1.0 if where == "s" else 2.0 ** -40)
    lora_b = one_rank_each(n, rank, adapters) * 2.0 ** -20
    p = operands(m, n, k, rank, adapters, x, lora_a, lora_b)
    got = qk.w8a8_lora_gemm(**p, out_dtype=torch.float32).double().cpu()
    ids = p["adapter_ids"].cpu().long()
    want = (big.double() * float(lora_a[0, 0, 0]))[:, None] * lora_b.double().sum(2)[ids]
    assert float(((got - want) / want).abs().max()) <= EXACT


@pytest.mark.parametrize("m,n,k,rank", [(6, 136, 272, 16), (64, 136, 528, 72), (70, 136, 272, 16), (140, 136, 80, 32),
                                        (90, 136, 272, 64), (200, 136, 272, 128)])
@pytest.mark.parametrize("where", ["token", "bf16 token", "scale"])
def test_infinities_as_the_formula_has_them(m, n, k, rank, where):
    """An infinite token element or lora_scale: infinity where all products have one sign, NaN where the formula
    has a difference of infinities or 0 times one; and rows that have none as they were."""
    adapters = 3
    g = torch.Generator().manual_seed(m)
    x = 0.5 + torch.rand((m, k), generator=g)
    la = 0.5 + torch.rand((adapters, rank, k), generator=g)
    lb = 0.5 + torch.rand((adapters, n, rank), generator=g)
    lb[:, 1::3, 2] *= -1.0       # a difference of infinities
    lb[:, 2::3, 5] = 0.0         # 0 times infinity
    dt = torch.bfloat16 if where == "bf16 token" else torch.float32
    scale = torch.tensor([1.0, 0.75, 0.5])
    clean = qk.w8a8_lora_gemm(**operands(m, n, k, rank, adapters, x.to(dt), la, lb, scale), out_dtype=torch.float32)
    hit = torch.zeros(m, dtype=torch.bool)
    if where == "scale":
        scale[1] = float("inf")
        hit = torch.arange(m) % adapters == 1
    else:
        hit[::4] = True
        x[hit, 7] = torch.tensor([float("inf"), -float("inf")])[torch.arange(int(hit.sum())) % 2]
    p = operands(m, n, k, rank, adapters, x.to(dt), la, lb, scale)
    got = qk.w8a8_lora_gemm(**p, out_dtype=torch.float32).cpu()
    ids = p["adapter_ids"].cpu().long()
    a64, b64 = p["lora_a"].double().cpu(), p["lora_b"].double().cpu()
    s = torch.einsum("ik,irk->ir", p["x"].double().cpu(), a64[ids]) * scale.double()[ids][:, None]
    want = (s[:, None] * b64[ids]).sum(2)
    assert bool(want[hit].isinf().any()) and bool(want[hit].isnan().any()) and not bool(want[hit].isfinite().any())
    assert torch.equal(got[hit].nan_to_num(0.5), want[hit].float().nan_to_num(0.5))
    assert torch.equal(got[~hit], clean.cpu()[~hit])
