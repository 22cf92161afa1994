"""Host-side tests (nothing is launched): what the layer operators answer beyond their limits."""
import ctypes

import pytest

from w8a8_int8_quantized_qk_b200 import build as qkbuild
from w8a8_int8_quantized_qk_b200 import qk

P = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails its checks first


@pytest.fixture(scope="module", autouse=True)
def L():
    qkbuild.build()
    return qk.lib()


def moe(m=4, hidden=32, inter=48, experts=3, topk=2):
    return qk.qk_w8a8_moe_layer(m, hidden, inter, experts, topk, P, P, P, P, P, P, P, P, P, qk.QK_BF16, P, 1 << 30, None)


@pytest.mark.parametrize("kw", [dict(experts=1 << 20, hidden=133136), dict(experts=1 << 14, inter=133136),
                                dict(experts=(1 << 31) - 1), dict(experts=1025, inter=133136, hidden=133136),
                                dict(m=65, experts=1 << 20, inter=133136), dict(topk=33, experts=1 << 14, inter=133136)])
def test_too_many_experts_slots_or_tokens(kw):
    """Whatever the other sizes are."""
    assert moe(**kw) == qk.QK_ERR_UNSUPPORTED
    sizes = {**dict(m=4, hidden=32, inter=48, experts=3, topk=2), **kw}
    assert qk.qk_w8a8_moe_layer_workspace_size(sizes["m"], sizes["hidden"], sizes["inter"], sizes["experts"],
                                               sizes["topk"]) == 0


@pytest.mark.parametrize("kw", [dict(experts=1 << 20, hidden=133152), dict(m=65, inter=133152)])
def test_too_long_rows_come_first(kw):
    assert moe(**kw) == qk.QK_ERR_OVERFLOW_BOUND


@pytest.mark.parametrize("kw", [dict(experts=1 << 20, hidden=133136, inter=40), dict(m=-1, experts=1 << 20),
                                dict(m=65, topk=0)])
def test_invalid_sizes_come_first(kw):
    assert moe(**kw) == qk.QK_ERR_INVALID_ARG
