"""Host-side tests (nothing is launched) of the operators around the linear layer: the fused norm and
quantiser, the projection with adapters, the MoE layer for a few tokens.  Argument checks come before
the device is touched, workspace queries answer 0 for what the call would reject, and the torch helpers
refuse host tensors."""
import ctypes

import pytest

from w8a8_int8_quantized_qk_b200 import build as qkbuild
from w8a8_int8_quantized_qk_b200 import qk

NULL = None
P16 = ctypes.c_void_p(0x1000)   # never dereferenced: every call below fails its checks first
P8 = ctypes.c_void_p(0x1008)    # 8-byte aligned only
P2 = ctypes.c_void_p(0x1002)
Q16 = ctypes.c_void_p(0x2000)


@pytest.fixture(scope="module", autouse=True)
def L():
    qkbuild.build()
    return qk.lib()


def _norm(fp8, m=4, k=32, x=P16, ldx=32, res=Q16, ldr=32, dt=qk.QK_BF16, w=P16, eps=1e-6, ro=NULL, ldo=32,
          y=NULL, ub=NULL, q=P16, s=P16):
    if fp8:
        return qk.qk_add_rmsnorm_quant_per_token_fp8(m, k, x, ldx, res, ldr, dt, w, eps, ro, ldo, y, ub, q, s, NULL)
    return qk.qk_add_rmsnorm_quant_per_token(m, k, x, ldx, res, ldr, dt, w, eps, ro, ldo, y, q, s, NULL)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,expect", [
    (dict(m=-1), qk.QK_ERR_INVALID_ARG),
    (dict(k=0), qk.QK_ERR_INVALID_ARG),
    (dict(k=24), qk.QK_ERR_INVALID_ARG),
    (dict(dt=7), qk.QK_ERR_INVALID_ARG),
    (dict(eps=0.0), qk.QK_ERR_INVALID_ARG),
    (dict(eps=-1e-6), qk.QK_ERR_INVALID_ARG),
    (dict(eps=float("nan")), qk.QK_ERR_INVALID_ARG),
    (dict(eps=float("inf")), qk.QK_ERR_INVALID_ARG),
    (dict(eps=1e-60), qk.QK_ERR_INVALID_ARG),                      # zero in binary32
    (dict(ldx=31), qk.QK_ERR_INVALID_ARG),
    (dict(ldr=16), qk.QK_ERR_INVALID_ARG),
    (dict(ro=Q16, ldo=16), qk.QK_ERR_INVALID_ARG),
    (dict(x=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(w=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(q=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(s=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(res=NULL, ro=Q16), qk.QK_ERR_INVALID_ARG),               # nothing to add
    (dict(ro=Q16, ldo=40), qk.QK_ERR_INVALID_ARG),                 # in place on other rows
    (dict(ro=P16, ldo=40), qk.QK_ERR_INVALID_ARG),
    (dict(x=P8), qk.QK_ERR_MISALIGNED),
    (dict(res=P8), qk.QK_ERR_MISALIGNED),
    (dict(w=P8), qk.QK_ERR_MISALIGNED),
    (dict(ro=P8), qk.QK_ERR_MISALIGNED),
    (dict(y=P8), qk.QK_ERR_MISALIGNED),
    (dict(q=P8), qk.QK_ERR_MISALIGNED),
    (dict(s=P2), qk.QK_ERR_MISALIGNED),
    (dict(ldx=36), qk.QK_ERR_MISALIGNED),                          # 72-byte rows
    (dict(ldr=36), qk.QK_ERR_MISALIGNED),
    (dict(m=0, x=NULL, res=NULL, w=NULL, q=NULL, s=NULL), qk.QK_OK),
])
def test_norm_rejects(fp8, kw, expect):
    assert _norm(fp8, **kw) == expect


def test_norm_bound_alignment():
    assert _norm(True, ub=P2) == qk.QK_ERR_MISALIGNED


def _lora(m=4, n=16, k=32, a=P16, b=P16, sa=P16, sw=P16, x=P16, xdt=qk.QK_BF16, ad=2, rank=8, la=P16, lb=P16,
          ls=NULL, ids=P16, out=P16, dt=qk.QK_BF16, ws=P16, wsb=1 << 30):
    return qk.qk_w8a8_lora_gemm(m, n, k, a, b, sa, sw, 1.0, x, xdt, ad, rank, la, lb, ls, ids, out, dt, ws, wsb, NULL)


@pytest.mark.parametrize("kw,expect", [
    (dict(m=-1), qk.QK_ERR_INVALID_ARG),
    (dict(n=-8), qk.QK_ERR_INVALID_ARG),
    (dict(n=12), qk.QK_ERR_INVALID_ARG),
    (dict(k=0), qk.QK_ERR_INVALID_ARG),
    (dict(k=40), qk.QK_ERR_INVALID_ARG),
    (dict(k=133152), qk.QK_ERR_OVERFLOW_BOUND),
    (dict(n=65535 * 256 + 8), qk.QK_ERR_UNSUPPORTED),
    (dict(m=(1 << 20) + 1), qk.QK_ERR_UNSUPPORTED),
    (dict(ad=(1 << 20) + 1), qk.QK_ERR_UNSUPPORTED),
    (dict(rank=0), qk.QK_ERR_INVALID_ARG),
    (dict(rank=12), qk.QK_ERR_INVALID_ARG),
    (dict(rank=136), qk.QK_ERR_INVALID_ARG),
    (dict(ad=0), qk.QK_ERR_INVALID_ARG),
    (dict(xdt=3), qk.QK_ERR_INVALID_ARG),
    (dict(dt=3), qk.QK_ERR_INVALID_ARG),
    (dict(a=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(b=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(sa=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(sw=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(x=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(la=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(lb=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(ids=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(out=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(a=P8), qk.QK_ERR_MISALIGNED),
    (dict(b=P8), qk.QK_ERR_MISALIGNED),
    (dict(sa=P8), qk.QK_ERR_MISALIGNED),
    (dict(sw=P8), qk.QK_ERR_MISALIGNED),
    (dict(x=P8), qk.QK_ERR_MISALIGNED),
    (dict(la=P8), qk.QK_ERR_MISALIGNED),
    (dict(lb=P8), qk.QK_ERR_MISALIGNED),
    (dict(ls=P2), qk.QK_ERR_MISALIGNED),
    (dict(ids=P2), qk.QK_ERR_MISALIGNED),
    (dict(out=P8), qk.QK_ERR_MISALIGNED),
    (dict(m=0), qk.QK_OK),
    (dict(n=0), qk.QK_OK),
])
def test_lora_rejects(kw, expect):
    assert _lora(**kw) == expect


def _moe(m=4, h=32, i=48, e=3, topk=2, a=P16, sa=P16, ids=P16, wt=P16, w13=P16, s13=P16, w2=P16, s2=P16, out=P16,
         dt=qk.QK_BF16, ws=P16, wsb=1 << 30):
    return qk.qk_w8a8_moe_layer(m, h, i, e, topk, a, sa, ids, wt, w13, s13, w2, s2, out, dt, ws, wsb, NULL)


@pytest.mark.parametrize("kw,expect", [
    (dict(m=-1), qk.QK_ERR_INVALID_ARG),
    (dict(h=0), qk.QK_ERR_INVALID_ARG),
    (dict(h=40), qk.QK_ERR_INVALID_ARG),
    (dict(i=0), qk.QK_ERR_INVALID_ARG),
    (dict(i=24), qk.QK_ERR_INVALID_ARG),
    (dict(e=0), qk.QK_ERR_INVALID_ARG),
    (dict(topk=0), qk.QK_ERR_INVALID_ARG),
    (dict(dt=9), qk.QK_ERR_INVALID_ARG),
    (dict(h=133152), qk.QK_ERR_OVERFLOW_BOUND),
    (dict(i=133152), qk.QK_ERR_OVERFLOW_BOUND),
    (dict(m=65), qk.QK_ERR_UNSUPPORTED),
    (dict(topk=33), qk.QK_ERR_UNSUPPORTED),
    (dict(e=1025), qk.QK_ERR_UNSUPPORTED),
    (dict(e=1024, i=1 << 20), qk.QK_ERR_OVERFLOW_BOUND),
    (dict(a=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(sa=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(ids=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(wt=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(w13=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(s13=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(w2=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(s2=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(out=NULL), qk.QK_ERR_INVALID_ARG),
    (dict(a=P8), qk.QK_ERR_MISALIGNED),
    (dict(w13=P8), qk.QK_ERR_MISALIGNED),
    (dict(w2=P8), qk.QK_ERR_MISALIGNED),
    (dict(out=P8), qk.QK_ERR_MISALIGNED),
    (dict(sa=P2), qk.QK_ERR_MISALIGNED),
    (dict(ids=P2), qk.QK_ERR_MISALIGNED),
    (dict(wt=P2), qk.QK_ERR_MISALIGNED),
    (dict(s13=P8), qk.QK_ERR_MISALIGNED),
    (dict(s2=P8), qk.QK_ERR_MISALIGNED),
    (dict(m=0), qk.QK_OK),
])
def test_moe_layer_rejects(kw, expect):
    assert _moe(**kw) == expect


def test_workspace_queries():
    for bad in ((0, 16, 32, 8), (4, 0, 32, 8), (4, 12, 32, 8), (4, 16, 40, 8), (4, 16, 32, 4), (4, 16, 32, 200),
                (4, 16, 133152, 8)):
        assert qk.qk_w8a8_lora_gemm_workspace_size(*bad) == 0
    for bad in ((0, 32, 48, 3, 2), (65, 32, 48, 3, 2), (4, 40, 48, 3, 2), (4, 32, 24, 3, 2), (4, 32, 48, 0, 2),
                (4, 32, 48, 3, 0), (4, 32, 48, 3, 33), (4, 32, 48, 1025, 2)):
        assert qk.qk_w8a8_moe_layer_workspace_size(*bad) == 0


def test_helpers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    a = torch.zeros((4, 16), dtype=torch.int8)
    s4, s8 = torch.ones(4), torch.ones(8)
    ad = torch.zeros((1, 8, 16), dtype=torch.bfloat16)
    bd = torch.zeros((1, 8, 8), dtype=torch.bfloat16)
    ids = torch.zeros((4, 1), dtype=torch.int32)
    w13 = torch.zeros((1, 32, 16), dtype=torch.int8)
    w2 = torch.zeros((1, 16, 16), dtype=torch.int8)
    for call in (lambda: qk.add_rmsnorm_quant_per_token(x, x[0]),
                 lambda: qk.add_rmsnorm_quant_per_token_fp8(x, x[0], x),
                 lambda: qk.w8a8_lora_gemm(a, a[:2], s4, s8, x, ad, bd, ids[:, 0]),
                 lambda: qk.w8a8_moe_layer(a, s4, ids, ids.float(), w13, torch.ones((1, 32)), w2,
                                           torch.ones((1, 16)))):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()
