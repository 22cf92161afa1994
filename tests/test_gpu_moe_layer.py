"""GPU tests of the MoE layer for a few tokens.

Bit for bit against the CPU oracle's pieces (INT8 GEMM and per-channel epilogue, SiLU quantiser), put
together pair by pair, with the weighted sum as fused multiply-adds over the slots in order (formed in 64 bits
and rounded: the product of two binary32 values is exact there).  And against the formula in 64 bits, where a
value of h that lies within the arithmetic's error of a rounding border may land on either side of it."""
import numpy as np
import pytest

from gpu_util import assert_bits, dev, host, need_gpu
from oracle.oracle import Oracle
from w8a8_int8_quantized_qk_b200 import qk, synth

pytestmark = pytest.mark.gpu

import torch  # noqa: E402


@pytest.fixture(scope="module")
def O():
    need_gpu()
    return Oracle(nthreads=8)


def make(m, experts, topk, hidden, inter, seed, ids=None):
    r = synth.streams(seed, ["a", "w13", "w2", "s", "ids", "wt"])
    p = dict(a=synth.int8_uniform(r["a"], (m, hidden)), w13=synth.int8_uniform(r["w13"], (experts, 2 * inter, hidden)),
             w2=synth.int8_uniform(r["w2"], (experts, hidden, inter)),
             sa=synth.scales_uniform(r["s"], (m,), 0.005, 0.03),
             s13=(synth.scales_uniform(r["s"], (experts, 2 * inter), 0.5, 1.5) / (73 * hidden ** 0.5)).astype(np.float32),
             s2=(synth.scales_uniform(r["s"], (experts, hidden), 0.5, 1.5) / (73 * inter ** 0.5)).astype(np.float32))
    p["ids"] = (np.argsort(r["ids"].random((m, experts)), 1)[:, :topk] if ids is None else ids).astype(np.int32)
    p["wt"] = r["wt"].random(p["ids"].shape).astype(np.float32)
    return p


def call(p, dt=torch.bfloat16, **kw):
    d = {n: dev(v) for n, v in p.items()}
    return qk.w8a8_moe_layer(d["a"], d["sa"], d["ids"], d["wt"], d["w13"], d["s13"], d["w2"], d["s2"], dt, **kw)


def reference(O, p):
    m, topk = p["ids"].shape
    hidden, inter, experts = p["a"].shape[1], p["w2"].shape[2], p["w2"].shape[0]
    out = np.zeros((m, hidden), np.float32)
    ys = np.zeros((m, topk, hidden), np.float32)
    for e in range(experts):
        t, s = np.nonzero(p["ids"] == e)
        if not len(t):
            continue
        gu = O.linear_from_q(p["a"][t], p["sa"][t], p["w13"][e], p["s13"][e])["out_f32"]
        q, sh = O.silu_mul_quant_per_token(np.ascontiguousarray(gu[:, :inter]), np.ascontiguousarray(gu[:, inter:]))
        ys[t, s] = O.linear_from_q(q, sh, p["w2"][e], p["s2"][e])["out_f32"]
    for s in range(topk):
        use = ((p["ids"][:, s] >= 0) & (p["ids"][:, s] < experts))[:, None]
        f = (p["wt"][:, s, None].astype(np.float64) * ys[:, s] + out).astype(np.float32)
        out = np.where(use, f, out)
    return out


def check(O, p):
    ref = reference(O, p)
    assert_bits(host(call(p, torch.float32)), ref, "out fp32")
    assert_bits(host(call(p)), O.f32_to_bf16(ref), "out bf16")
    assert qk.device_status() == qk.QK_OK


@pytest.mark.parametrize("m,experts,topk,hidden,inter", [
    (1, 1, 1, 16, 16), (1, 8, 2, 4096, 512), (2, 4, 2, 512, 1040), (3, 5, 3, 1040, 528), (4, 64, 6, 256, 176),
    (5, 3, 1, 2064, 48), (8, 2, 2, 528, 272), (9, 1, 1, 272, 528), (16, 16, 4, 512, 256), (17, 2, 1, 1024, 144),
    (33, 3, 2, 272, 1040), (64, 2, 2, 512, 528), (64, 128, 8, 64, 64), (40, 1, 1, 80, 4112), (2, 2, 2, 16400, 32),
    (3, 1000, 32, 32, 16), (6, 9, 4, 48, 14352)])
def test_moe_layer(O, m, experts, topk, hidden, inter):
    check(O, make(m, experts, topk, hidden, inter, seed=m + experts + hidden))


@pytest.mark.parametrize("m", [1, 6, 30])
@pytest.mark.parametrize("kind", ["none", "some", "same", "twice", "outside"])
def test_moe_layer_ids(O, m, kind):
    """Tokens without experts, all tokens on one expert, an expert twice in a token, ids out of range."""
    rng = np.random.default_rng(m)
    ids = {"none": np.full((m, 3), -1), "some": rng.integers(-1, 5, (m, 3)), "same": np.full((m, 3), 3),
           "twice": np.tile([1, 4, 1], (m, 1)),
           "outside": np.tile([5, 2 ** 31 - 1, -2 ** 31], (m, 1)) * (rng.random((m, 3)) < 0.7)}[kind]
    p = make(m, 5, 3, 272, 144, seed=m, ids=ids)
    if kind == "none":
        assert not host(call(p, torch.float32)).any()
    check(O, p)


def test_moe_layer_in_64_bits():
    """u = 2^-24: g and u carry three roundings each, silu its own few (4 steps) and the product one, so h is
    within 16 u relative (g's error passes silu with a factor of at most 1 + |g| e^-|g| < 1.4), v = h / sh within
    20 u * 127 < 2e-4 of a unit.  Codes nearer than that to a border may differ by one: each moves y by its
    weight times the scales.  The sums over slots and the output's rounding add 2^-8 in bf16, u in binary32."""
    need_gpu()
    p = make(12, 6, 2, 1040, 1056, seed=77)
    out = host(call(p, torch.float32)).astype(np.float64)
    m, topk = p["ids"].shape
    inter = p["w2"].shape[2]
    want, slack = np.zeros_like(out), np.zeros_like(out)
    for i in range(m):
        for s in range(topk):
            e = p["ids"][i, s]
            gu = (p["w13"][e].astype(np.float64) @ p["a"][i]) * p["sa"][i].astype(np.float64) * p["s13"][e]
            g, u = gu[:inter], gu[inter:]
            h = g / (1 + np.exp(-g)) * u
            sh = np.abs(h).max() / 127
            v = h / sh
            near = (np.abs(np.abs(v - np.floor(v)) - 0.5) < 2e-4).astype(np.float64)
            w2, s2 = p["w2"][e].astype(np.float64), p["s2"][e].astype(np.float64)
            y = (w2 @ np.rint(v)) * sh * s2
            want[i] += p["wt"][i, s] * y
            slack[i] += p["wt"][i, s] * ((np.abs(w2) @ near) * sh * s2 + 24 * 2.0 ** -24 * np.abs(y))
    slack += 4 * 2.0 ** -24 * np.abs(want) * topk
    # partial sums over the slots are rounded at their own size
    assert np.all(np.abs(out - want) <= slack + 8 * 2.0 ** -24 * np.abs(out).max())


def test_moe_layer_tokens_do_not_depend_on_the_batch():
    """A token's output is the same alone and in any company, in any order, and again."""
    need_gpu()
    p = make(24, 6, 2, 528, 272, seed=11)
    whole = call(p)
    assert torch.equal(call(p), whole)
    for i in (0, 7, 23):
        one = {n: (v[i:i + 1] if n in ("a", "sa", "ids", "wt") else v) for n, v in p.items()}
        assert torch.equal(call(one), whole[i:i + 1])
    back = {n: (np.ascontiguousarray(v[::-1]) if n in ("a", "sa", "ids", "wt") else v) for n, v in p.items()}
    assert torch.equal(call(back), whole.flip(0))


def test_moe_layer_unused_experts_and_slots():
    """What the scales of experts nobody uses, or the weights of slots without an expert, hold does not matter."""
    need_gpu()
    p = make(7, 5, 3, 272, 144, seed=4, ids=np.tile([1, -1, 3], (7, 1)))
    clean = call(p)
    p["s13"][[0, 2, 4]] = np.nan
    p["s2"][[0, 2, 4]] = np.inf
    p["wt"][:, 1] = np.nan
    assert torch.equal(call(p), clean)


@pytest.mark.parametrize("m", [1, 20])
def test_moe_layer_workspace(m):
    need_gpu()
    p = make(m, 4, 2, 512, 272, seed=m)
    first = call(p)
    need = qk.qk_w8a8_moe_layer_workspace_size(m, 512, 272, 4, 2)
    for fill in (0, 255, 127):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        buf = torch.full((m + 2, 512), 3.0, dtype=torch.bfloat16, device="cuda")
        out = call(p, out=buf[:m], workspace=ws[:need])
        assert torch.equal(out, first)
        assert bool((buf[m:] == 3.0).all()) and bool((ws[need:] == fill).all())
    with pytest.raises(qk.QKError):
        call(p, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


def test_moe_layer_helper_refusals():
    need_gpu()
    p = {n: dev(v) for n, v in make(4, 3, 2, 64, 48, seed=1).items()}
    args = [p[n] for n in ("a", "sa", "ids", "wt", "w13", "s13", "w2", "s2")]
    qk.w8a8_moe_layer(*args)
    for at, bad in ((0, p["a"].float()), (1, p["sa"][:2]), (2, p["ids"].long()), (2, p["ids"][:2]),
                    (3, p["wt"].double()), (3, p["wt"][:, :1]), (4, p["w13"][:, :48]), (5, p["s13"][:1]),
                    (6, p["w2"][0]), (6, p["w2"].transpose(1, 2)), (7, p["s2"][:, :8])):
        with pytest.raises(ValueError):
            qk.w8a8_moe_layer(*[bad if j == at else v for j, v in enumerate(args)])
    with pytest.raises(TypeError):
        qk.w8a8_moe_layer(*args, out_dtype=torch.float16)
    with pytest.raises(qk.QKError):
        qk.w8a8_moe_layer(*[torch.cat([v] * 17) if j < 4 else v for j, v in enumerate(args)])  # 68 tokens
    empty = [v[:0] if j < 4 else v for j, v in enumerate(args)]
    assert qk.w8a8_moe_layer(*empty).shape == (0, 64)
