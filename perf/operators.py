"""The operators around the W8A8 linear layer, as a serving program calls them: their cases, inputs,
plain forms and results in 64 bits.

Three operators of one decoder layer:

* ``norm`` -- residual addition, root-mean-square norm and per-token 8-bit quantisation: it makes the
  int8 (or e4m3) tokens and scales that the layer's products read;
* ``lora`` -- the shared W8A8 projection with the low-rank adapters of many requests beside it;
* ``moe``  -- a whole mixture-of-experts layer (gate and up, SiLU, down, weighted sum) for a few tokens.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the library's kernels.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_T = {BF16: torch.bfloat16, F32: torch.float32}
_SIZE = {BF16: 2, F32: 4}


# ------------------------------------------------------------------ cases
def _norm(m, k, x=BF16, out="int8", residual=True, norm_out=False, bound=False, name=None):
    c = dict(op="norm", m=m, k=k, x=x, out=out, residual=residual, norm_out=norm_out, bound=bound)
    return dict(c, name=name) if name else c


def _lora(m, n, k, rank, adapters, x=BF16, out=BF16, grouped=False, name=None):
    c = dict(op="lora", m=m, n=n, k=k, rank=rank, adapters=adapters, x=x, out=out, grouped=grouped)
    return dict(c, name=name) if name else c


def _moe(m, experts, topk, hidden, inter, out=BF16, local=False, name=None):
    c = dict(op="moe", m=m, experts=experts, topk=topk, hidden=hidden, inter=inter, out=out, local=local)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence being decoded: latency is all that counts
        _norm(1, 4096, name="norm_one_token"),
        # a decode batch; the normalised tokens are also kept for adapters and a router
        _norm(64, 8192, norm_out=True, name="norm_decode_batch"),
        # a prompt of the prefill workload's size
        _norm(4096, 4096, name="norm_prompt"),
        # first norm of a model (no residual yet), fp32 stream, e4m3 with a bounded scale, odd sizes
        _norm(2049, 8208, x=F32, out="fp8", residual=False, bound=True, name="norm_f32_fp8_odd"),
        # the decode workload's projection with an adapter for every request
        _lora(4, 14336, 4096, 16, 4, name="lora_decode"),
        # a larger decode batch, requests of many adapters in any order, some without one
        _lora(64, 4096, 4096, 64, 32, name="lora_decode_batch"),
        # the prefill workload's projection: the tokens of a request lie together
        _lora(4096, 4096, 4096, 16, 4, grouped=True, name="lora_prompt"),
        # fp32 activations and output, sizes that fill no tile
        _lora(37, 1032, 2064, 8, 5, x=F32, out=F32, name="lora_f32_odd"),
        # one token through two of eight large experts: a stream of weights
        _moe(1, 8, 2, 4096, 14336, name="moe_one_token"),
        # a few tokens over many small experts
        _moe(4, 64, 6, 2048, 1408, name="moe_small_experts"),
        # a batch that keeps every expert busy
        _moe(32, 8, 2, 4096, 14336, name="moe_batch"),
        # experts spread over ranks: the slots of other ranks' experts are marked -1; odd sizes
        _moe(7, 5, 3, 1040, 528, local=True, name="moe_local_odd"),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], even over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return int(min(hi, max(lo, step * round(v / step))))


def draw(rng):
    op = rng.choice(("norm", "lora", "moe"))
    if op == "norm":
        k = _log_int(rng, 64, 16384, 16)
        m = _log_int(rng, 1, min(8192, max(1, (1 << 24) // k)))
        return _norm(m, k, x=rng.choice((BF16, BF16, F32)), out=rng.choice(("int8", "int8", "fp8")),
                     residual=rng.random() < 0.7, norm_out=rng.random() < 0.3, bound=rng.random() < 0.3)
    if op == "lora":
        n, k, rank = _log_int(rng, 256, 14336, 8), _log_int(rng, 256, 8192, 16), 8 * rng.randint(1, 16)
        m = _log_int(rng, 1, min(4096, (1 << 33) // (n * k) * 4 + 1, (1 << 29) // (rank * (n + k)) + 1))
        return _lora(m, n, k, rank, rng.randint(1, 24), x=rng.choice((BF16, BF16, F32)),
                     out=rng.choice((BF16, BF16, F32)), grouped=rng.random() < 0.5)
    hidden, inter = _log_int(rng, 512, 4096, 16), _log_int(rng, 256, 8192, 16)
    experts = _log_int(rng, 1, max(1, min(128, (1 << 30) // (3 * hidden * inter))))
    return _moe(_log_int(rng, 1, 64), experts, rng.randint(1, min(8, experts)), hidden, inter,
                local=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _activations(g, m, k):
    """N(0, 1) with 1 % of the columns twenty times as large, as the decode workload has them."""
    x = _randn(g, m, k)
    at = torch.randperm(k, generator=g, device="cuda")[: max(1, round(0.01 * k))]
    x[:, at] *= 20.0
    return x


def _weights(g, *shape):
    """int8 weights and per-channel scales that keep the products' size near one."""
    w = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
    s = (0.5 + torch.rand(shape[:-1], generator=g, device="cuda")) / (73.0 * math.sqrt(shape[-1]))
    return w, s


def _tokens(x):
    """Per-token int8: the codes and the scales."""
    s = x.float().abs().amax(1).clamp_min(1e-12) / 127.0
    return torch.round(x.float() * (1.0 / s)[:, None]).to(torch.int8), s


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "norm":
        m, k, t = case["m"], case["k"], _T[case["x"]]
        s["xs"] = _activations(g, m, k).to(t)
        s["weight"] = (1.0 + 0.2 * _randn(g, k)).to(t)
        s["res"] = (2.0 * _activations(g, m, k)).to(t) if case["residual"] else None
        # a bound that some rows' scales pass
        s["ub"] = torch.full((1,), 24.0 / 448.0, device="cuda") if case["bound"] and case["out"] == "fp8" else None
        s["eps"] = 1e-6
    elif case["op"] == "lora":
        m, n, k, r, ad = (case[v] for v in ("m", "n", "k", "rank", "adapters"))
        s["xs"] = _activations(g, m, k).to(_T[case["x"]])
        s["a"], s["sa"] = _tokens(s["xs"])
        s["w"], s["sw"] = _weights(g, n, k)
        s["lora_a"] = (_randn(g, ad, r, k) / math.sqrt(k)).bfloat16()
        s["lora_b"] = (_randn(g, ad, n, r) / math.sqrt(r)).bfloat16()
        s["lora_scale"] = 0.25 + torch.rand(ad, generator=g, device="cuda")
        ids = torch.randint(-1, ad, (m,), generator=g, device="cuda", dtype=torch.int32)
        s["ids"] = torch.sort(ids).values if case["grouped"] else ids
    else:
        m, e, topk, h, i = (case[v] for v in ("m", "experts", "topk", "hidden", "inter"))
        s["a"], s["sa"] = _tokens(_activations(g, m, h).bfloat16())
        s["w13"], s["s13"] = _weights(g, e, 2 * i, h)
        s["w2"], s["s2"] = _weights(g, e, h, i)
        top = torch.topk(_randn(g, m, e), topk, dim=1)
        s["weights"], s["ids"] = torch.softmax(top.values, 1), top.indices.to(torch.int32)
        if case["local"]:
            away = torch.rand((m, topk), generator=g, device="cuda") < 0.5
            s["ids"] = torch.where(away, torch.full_like(s["ids"], -1), s["ids"])
    return s


# ------------------------------------------------------------------ one pass
def _plain_norm(s):
    r = s["xs"] if s["res"] is None else (s["xs"].float() + s["res"].float()).to(s["xs"].dtype)
    f, qmax = r.float(), 127.0 if s["out"] == "int8" else 448.0
    t = f * s["weight"].float()
    amax = t.abs().amax(1)
    rstd = torch.rsqrt((f * f).mean(1) + s["eps"])
    z = amax * rstd
    whole = z.clamp_min(1e-12) / qmax
    scale = whole if s["ub"] is None else torch.minimum(whole, s["ub"])
    # t / amax fills the range exactly; a clamped or bounded scale takes the norm's factor instead
    inv = torch.where((scale == whole) & (z >= 1e-12), qmax / amax, rstd / scale)
    v = (t * inv[:, None]).clamp(-qmax, qmax)
    q = torch.round(v).to(torch.int8) if s["out"] == "int8" else v.to(torch.float8_e4m3fn)
    out = {"q": q, "scale": scale}
    if s["res"] is not None:
        out["residual"] = r
    if s["norm_out"]:
        out["norm"] = (t * rstd[:, None]).to(s["xs"].dtype)
    return out


def _plain_lora(s):
    base = (s["a"].float() @ s["w"].float().T) * s["sa"][:, None] * s["sw"]
    used = (s["ids"] >= 0)[:, None]
    at = s["ids"].clamp_min(0).long()
    low = torch.bmm(s["lora_a"][at].float(), s["xs"].float()[:, :, None]) * s["lora_scale"][at][:, None, None]
    delta = torch.bmm(s["lora_b"][at].float(), low)[:, :, 0]
    return torch.where(used, base + delta, base).to(_T[s["out"]])


def _plain_moe(s):
    i, at = s["inter"], s["ids"].clamp_min(0).long()
    rows = torch.arange(s["m"], device="cuda")[:, None]
    every = torch.matmul(s["a"].float(), s["w13"].float().transpose(1, 2)) * s["s13"][:, None]  # [E, m, 2I]
    gu = every[at, rows] * s["sa"][:, None, None]  # [m, topk, 2I]
    gate, up = gu[..., :i], gu[..., i:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    sh = h.abs().amax(2).clamp_min(1e-12) / 127.0
    q = torch.round(h * (1.0 / sh)[..., None])
    # every expert's tokens at their own places, so that one product over the experts serves them all
    spread = torch.zeros((s["experts"], s["m"], s["topk"], i), device="cuda")
    slots = torch.arange(s["topk"], device="cuda")[None]
    spread[at, rows, slots] = q
    y = torch.matmul(spread.flatten(1, 2), s["w2"].float().transpose(1, 2)).unflatten(1, (s["m"], s["topk"]))
    y = y[at, rows, slots] * sh[..., None] * s["s2"][at]
    return (y * (s["weights"] * (s["ids"] >= 0))[..., None]).sum(1).to(_T[s["out"]])


def _own(s):
    from w8a8_int8_quantized_qk_b200 import qk

    if s["op"] == "norm":
        if s["out"] == "int8":
            q, scale, residual, norm = qk.add_rmsnorm_quant_per_token(
                s["xs"], s["weight"], s["res"], s["eps"], want_norm=s["norm_out"])
        else:
            q, scale, residual, norm = qk.add_rmsnorm_quant_per_token_fp8(
                s["xs"], s["weight"], s["res"], s["eps"], scale_ub=s["ub"], want_norm=s["norm_out"])
            q = q.view(torch.float8_e4m3fn)
        out = {"q": q, "scale": scale, "residual": residual, "norm": norm}
        return {name: v for name, v in out.items() if v is not None}
    if s["op"] == "lora":
        return qk.w8a8_lora_gemm(s["a"], s["w"], s["sa"], s["sw"], s["xs"], s["lora_a"], s["lora_b"], s["ids"],
                                 s["lora_scale"], out_dtype=_T[s["out"]])
    return qk.w8a8_moe_layer(s["a"], s["sa"], s["ids"], s["weights"], s["w13"], s["s13"], s["w2"], s["s2"],
                             out_dtype=_T[s["out"]])


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "lora": _plain_lora, "moe": _plain_moe}[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "norm":
        m, k, es = case["m"], case["k"], _SIZE[case["x"]]
        tensors = 1 + 2 * case["residual"] + case["norm_out"]
        return {"bytes": m * k * (tensors * es + 1) + k * es + 4 * m, "flops": 8 * m * k}
    if case["op"] == "lora":
        m, n, k, r = case["m"], case["n"], case["k"], case["rank"]
        used = min(m, case["adapters"])
        size = (m * k * (1 + _SIZE[case["x"]]) + n * k + 4 * (m + n) + used * r * (n + k) * 2
                + m * n * _SIZE[case["out"]])
        return {"bytes": size, "flops": 2 * m * n * k + 2 * m * r * (n + k)}
    m, e, topk, h, i = (case[v] for v in ("m", "experts", "topk", "hidden", "inter"))
    pairs = m * topk * (0.5 if case["local"] else 1.0)
    # the experts that so many uniform choices are expected to meet
    active = e * (1.0 - (1.0 - 1.0 / e) ** pairs) if pairs < 4 * e else e
    size = active * (3 * h * i + 4 * (2 * i + h)) + m * h * (1 + _SIZE[case["out"]])
    return {"bytes": size, "flops": 2 * pairs * 3 * h * i}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_norm(s):
    rows = s["xs"].double()
    if s["res"] is not None:
        rows = (rows + s["res"].double()).to(s["xs"].dtype).double()
    weighted = rows * s["weight"].double()[None, :]
    unit = 1.0 / torch.sqrt(rows.square().sum(1) / s["k"] + s["eps"])
    normal = weighted * unit[:, None]
    top = 127.0 if s["out"] == "int8" else 448.0
    scale = torch.maximum(normal.abs().max(1).values, torch.tensor(1e-12, device="cuda", dtype=torch.float64)) / top
    if s["ub"] is not None:
        scale = torch.minimum(scale, s["ub"].double())
    codes = normal / scale[:, None]
    if s["out"] == "int8":
        codes = None  # whole numbers: compared with the plain form's alone
    else:
        codes = torch.clamp(codes, -448.0, 448.0)
    out = {"q": codes, "scale": scale}
    if s["res"] is not None:
        out["residual"] = rows
    if s["norm_out"]:
        out["norm"] = normal
    return out


def _exact_lora(s):
    out = (s["a"].double() * s["sa"].double()[:, None]) @ (s["w"].double() * s["sw"].double()[:, None]).T
    x, ids = s["xs"].double(), s["ids"].tolist()
    for adapter in set(ids) - {-1}:
        rows = torch.tensor([j for j, v in enumerate(ids) if v == adapter], device="cuda")
        product = s["lora_b"][adapter].double() @ s["lora_a"][adapter].double()
        out[rows] += s["lora_scale"][adapter].double() * (x[rows] @ product.T)
    return out


def _exact_moe(s):
    out = torch.zeros((s["m"], s["hidden"]), device="cuda", dtype=torch.float64)
    tokens = s["a"].double() * s["sa"].double()[:, None]
    for expert in set(s["ids"].flatten().tolist()) - {-1}:
        token, slot = torch.nonzero(s["ids"] == expert, as_tuple=True)
        both = tokens[token] @ (s["w13"][expert].double() * s["s13"][expert].double()[:, None]).T
        h = torch.nn.functional.silu(both[:, : s["inter"]]) * both[:, s["inter"]:]
        step = torch.clamp_min(h.abs().max(1, keepdim=True).values, 1e-12) / 127.0
        y = (torch.round(h / step) * step) @ (s["w2"][expert].double() * s["s2"][expert].double()[:, None]).T
        out.index_add_(0, token, y * s["weights"][token, slot].double()[:, None])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "lora": _exact_lora, "moe": _exact_moe}[case["op"]](s)
