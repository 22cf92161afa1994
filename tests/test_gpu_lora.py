"""GPU tests of the W8A8 projection with adapters beside it.

Rows without an adapter equal qk_w8a8_gemm bit for bit.  Rows with one are held to the formula in 64 bits:
with u = 2^-24 the base is three roundings, (1 + u)^3; s and d are binary32 sums of k and rank products,
each within its count of additions plus two roundings (and one for lora_scale) times the sum of the
products' magnitudes; the last addition and the rounding to the output's type follow (bf16 2^-8, binary32 u)."""
import numpy as np
import pytest

from gpu_util import need_gpu
from w8a8_int8_quantized_qk_b200 import qk

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

U = 2.0 ** -24


def make(m, n, k, rank, adapters, x_dtype, seed, ids=None, scaled=True):
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=g, device="cuda")

    x = randn(m, k).to(x_dtype)
    a, sa = qk.quantize_per_token(x)
    b = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    sw = (0.5 + torch.rand(n, generator=g, device="cuda")) / (73.0 * k ** 0.5)
    la = (randn(adapters, rank, k) / k ** 0.5).bfloat16()
    lb = (randn(adapters, n, rank) / rank ** 0.5).bfloat16()
    ls = 0.25 + torch.rand(adapters, generator=g, device="cuda") if scaled else None
    if ids is None:
        ids = torch.randint(-1, adapters, (m,), generator=g, device="cuda", dtype=torch.int32)
    return dict(a=a, b=b, scale_a=sa, scale_b=sw, x=x, lora_a=la, lora_b=lb, adapter_ids=ids, lora_scale=ls)


def check(p, out, alpha=1.0):
    a, b, x = p["a"].double(), p["b"].double(), p["x"].double()
    m, k = a.shape
    rank, adapters = p["lora_a"].shape[1], p["lora_a"].shape[0]
    base = (a @ b.T) * p["scale_a"].double()[:, None] * p["scale_b"].double() * float(np.float32(alpha))
    d, mag = torch.zeros_like(base), torch.zeros_like(base)
    for e in range(adapters):
        rows = (p["adapter_ids"] == e).nonzero()[:, 0]
        if not len(rows):
            continue
        la, lb = p["lora_a"][e].double(), p["lora_b"][e].double()
        ls = 1.0 if p["lora_scale"] is None else p["lora_scale"][e].double()
        d[rows] = ls * ((x[rows] @ la.T) @ lb.T)
        mag[rows] = ls * ((x[rows].abs() @ la.abs().T) @ lb.abs().T)
    want = base + d
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else U
    fp32 = 4 * U * base.abs() + (k + rank + 8) * U * mag + U * want.abs()
    assert bool(((out.double() - want).abs() <= fp32 + half * (want.abs() + fp32)).all())


def plain_rows(p, out, alpha, dt):
    """Rows without an adapter: the plain GEMM's bits."""
    ids = p["adapter_ids"]
    rows = ((ids < 0) | (ids >= p["lora_a"].shape[0])).nonzero()[:, 0]
    ref, _ = qk.w8a8_gemm(p["a"], p["b"], p["scale_a"], p["scale_b"], 0, alpha, dt)
    assert torch.equal(out[rows], ref[rows])


# decode sizes, both sides of every boundary between forms, ragged tiles, the split forms of the GEMM
@pytest.mark.parametrize("m,n,k,rank,adapters", [
    (1, 8, 16, 8, 1), (1, 4096, 4096, 16, 3), (2, 520, 1040, 8, 2), (4, 1024, 2064, 24, 4), (7, 264, 4112, 64, 3),
    (8, 2056, 512, 128, 9), (9, 1032, 1040, 16, 4), (16, 512, 4096, 40, 16), (17, 264, 272, 8, 5),
    (31, 4096, 512, 32, 40), (33, 1032, 2064, 8, 5), (64, 1024, 1040, 64, 7), (65, 136, 528, 128, 2),
    (128, 2048, 512, 16, 3), (129, 264, 272, 56, 4), (200, 1032, 4096, 16, 6), (300, 4096, 1024, 8, 2),
    (256, 1024, 14336, 16, 3), (700, 520, 528, 72, 11), (2304, 2304, 512, 16, 4),
    (1024, 264, 272, 8, 1200), (1025, 136, 144, 120, 2), (2500, 264, 144, 32, 70), (3000, 520, 80, 16, 1)])
@pytest.mark.parametrize("x_dtype,out_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                               (torch.bfloat16, torch.float32)])
def test_lora(m, n, k, rank, adapters, x_dtype, out_dtype):
    p = make(m, n, k, rank, adapters, x_dtype, seed=m + n + k)
    alpha = 0.75
    out = qk.w8a8_lora_gemm(**p, output_scale=alpha, out_dtype=out_dtype)
    check(p, out, alpha)
    plain_rows(p, out, alpha, out_dtype)
    assert qk.device_status() == qk.QK_OK


@pytest.mark.parametrize("m", [1, 5, 24, 150, 2100])
@pytest.mark.parametrize("kind", ["none", "one", "each", "outside", "grouped"])
def test_lora_ids(m, kind):
    adapters = max(m, 3)
    ids = {"none": torch.full((m,), -1), "one": torch.full((m,), 2), "each": torch.arange(m).flip(0),
           "outside": torch.tensor([adapters, -7, 1 << 30, -(1 << 31), 1])[torch.arange(m) % 5],
           "grouped": torch.arange(m) // 16}[kind].to(torch.int32).cuda()
    p = make(m, 1032, 528, 16, adapters, torch.bfloat16, seed=m, ids=ids, scaled=kind != "one")
    out = qk.w8a8_lora_gemm(**p)
    check(p, out)
    plain_rows(p, out, 1.0, torch.bfloat16)


@pytest.mark.parametrize("m", [3, 40, 300])
def test_lora_values_stay_with_their_rows(m):
    """What is not finite in an adapter, in a token or in a scale reaches the rows that use it and no other."""
    p = make(m, 520, 272, 16, 4, torch.bfloat16, seed=m)
    p["adapter_ids"] = (torch.arange(m, device="cuda") % 4 - 1).to(torch.int32)  # -1, 0, 1, 2: nobody uses 3
    clean = qk.w8a8_lora_gemm(**p)
    p["lora_a"][3] = float("nan")
    p["lora_b"][3] = float("inf")
    p["lora_b"][1] = float("nan")
    p["lora_scale"][0] = float("inf")
    p["x"][2, 5] = float("nan")
    dirty = qk.w8a8_lora_gemm(**p)
    keep = ((p["adapter_ids"] == 2) | (p["adapter_ids"] == -1))
    keep[2] = False
    assert torch.equal(clean[keep], dirty[keep])
    assert bool(dirty[p["adapter_ids"] == 1].isnan().all())


@pytest.mark.parametrize("m,n,k", [(4, 1024, 1024), (40, 1024, 1024), (300, 2304, 1024)])
def test_lora_repeats_and_workspace(m, n, k):
    """Any contents of the workspace, the same bits each time, nothing behind the outputs touched."""
    p = make(m, n, k, 16, 3, torch.bfloat16, seed=5)
    need = qk.qk_w8a8_lora_gemm_workspace_size(m, n, k, 16)
    first = qk.w8a8_lora_gemm(**p)
    for fill in (0, 255, 127):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        buf = torch.full((m + 2, n), 3.0, dtype=torch.bfloat16, device="cuda")
        out = qk.w8a8_lora_gemm(**p, out=buf[:m], workspace=ws[:need])
        assert torch.equal(out, first)
        assert bool((buf[m:] == 3.0).all()) and bool((ws[need:] == fill).all())
    with pytest.raises(qk.QKError):
        qk.w8a8_lora_gemm(**p, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


def test_lora_helper_refusals():
    p = make(4, 64, 64, 8, 2, torch.bfloat16, seed=1)
    qk.w8a8_lora_gemm(**p)
    for kw in (dict(lora_a=p["lora_a"].float()), dict(lora_b=p["lora_b"][:1]), dict(lora_a=p["lora_a"][0]),
               dict(adapter_ids=p["adapter_ids"].long()), dict(adapter_ids=p["adapter_ids"][:2]),
               dict(x=p["x"][:, ::2]), dict(x=p["x"][:2]), dict(scale_a=p["scale_a"][:2]),
               dict(lora_scale=p["lora_scale"].double()), dict(out=torch.empty((4, 32), device="cuda")),
               dict(b=p["b"].t()), dict(a=p["a"].float())):
        with pytest.raises(ValueError):
            qk.w8a8_lora_gemm(**{**p, **kw})
    with pytest.raises(TypeError):
        qk.w8a8_lora_gemm(**{**p, "x": p["x"].half()})
    with pytest.raises(TypeError):
        qk.w8a8_lora_gemm(**p, out_dtype=torch.float16)
    empty = {**p, "a": p["a"][:0], "x": p["x"][:0], "scale_a": p["scale_a"][:0], "adapter_ids": p["adapter_ids"][:0]}
    assert qk.w8a8_lora_gemm(**empty).shape == (0, 64)
