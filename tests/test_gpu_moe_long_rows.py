"""GPU tests of the MoE layer where a row of h is longer than a cluster's threads hold (inter above 32768) and waits
in the gate sums' place: bit for bit, as in the tests of the other sizes."""
import numpy as np
import pytest

from gpu_util import need_gpu
from oracle.oracle import Oracle
from test_gpu_moe_layer import call, check, make

pytestmark = pytest.mark.gpu

import torch  # noqa: E402


@pytest.fixture(scope="module")
def O():
    need_gpu()
    return Oracle(nthreads=8)


# one row block more than a cluster holds; the last size accepted; the longest row that stays in registers
@pytest.mark.parametrize("m,experts,topk,hidden,inter", [
    (1, 2, 1, 48, 32784), (3, 3, 2, 64, 40016), (64, 2, 1, 32, 32896), (2, 2, 2, 16, 133136), (2, 2, 2, 48, 32768)])
def test_long_rows(O, m, experts, topk, hidden, inter):
    check(O, make(m, experts, topk, hidden, inter, seed=m + experts + inter))


def test_long_rows_without_experts(O):
    ids = np.array([[-1, 1], [-1, -1], [1, 1]])
    p = make(3, 2, 2, 48, 33040, seed=5, ids=ids)
    check(O, p)
    first = call(p)
    assert all(torch.equal(call(p), first) for _ in range(5))
    assert not bool(first[1].any())
