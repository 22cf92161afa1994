"""GPU tests of the operators around the linear layer as they are used together: norm, projection with
adapters, norm, MoE layer, as one layer of a decoder runs them -- eagerly, captured and replayed, on other
streams, from several threads.  Each operator's values are held to their definitions in its own tests; here
the runs have to agree bit for bit with the calls made one by one."""
import threading

import pytest

from gpu_util import need_gpu
from w8a8_int8_quantized_qk_b200 import qk

pytestmark = pytest.mark.gpu

import torch  # noqa: E402

HIDDEN, INTER, EXPERTS, TOPK, ADAPTERS, RANK = 1040, 528, 6, 2, 3, 16


def weights(seed, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)

    def rand8(*s):
        return torch.randint(-127, 128, s, generator=g, device=device, dtype=torch.int8)

    def scale(*s):
        return (0.5 + torch.rand(s, generator=g, device=device)) / 2000.0

    def randn(*s):
        return torch.randn(s, generator=g, device=device)

    return dict(norm1=(1 + 0.1 * randn(HIDDEN)).bfloat16(), norm2=(1 + 0.1 * randn(HIDDEN)).bfloat16(),
                w=rand8(HIDDEN, HIDDEN), sw=scale(HIDDEN), la=(randn(ADAPTERS, RANK, HIDDEN) / 30).bfloat16(),
                lb=(randn(ADAPTERS, HIDDEN, RANK) / 4).bfloat16(), w13=rand8(EXPERTS, 2 * INTER, HIDDEN),
                s13=scale(EXPERTS, 2 * INTER), w2=rand8(EXPERTS, HIDDEN, INTER), s2=scale(EXPERTS, HIDDEN))


def tokens(m, seed, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return dict(x=torch.randn((m, HIDDEN), generator=g, device=device).bfloat16(),
                res=torch.randn((m, HIDDEN), generator=g, device=device).bfloat16(),
                ids=torch.randint(-1, ADAPTERS, (m,), generator=g, device=device, dtype=torch.int32),
                top=torch.randint(-1, EXPERTS, (m, TOPK), generator=g, device=device, dtype=torch.int32),
                wt=torch.rand((m, TOPK), generator=g, device=device))


def layer(w, t, stream=None):
    """The projection's output is the layer's next x; the residual is carried along in place."""
    res = t["res"].clone() if stream is None else t["res"]
    q, s, res, y = qk.add_rmsnorm_quant_per_token(t["x"], w["norm1"], res, want_norm=True,
                                                  residual_out=res if stream is None else None, stream=stream)
    h = qk.w8a8_lora_gemm(q, w["w"], s, w["sw"], y, w["la"], w["lb"], t["ids"], stream=stream)
    q, s, res, _ = qk.add_rmsnorm_quant_per_token(h, w["norm2"], res, stream=stream)
    out = qk.w8a8_moe_layer(q, s, t["top"], t["wt"], w["w13"], w["s13"], w["w2"], w["s2"], stream=stream)
    return out, res


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("m", [1, 5, 40, 64])
def test_chain_is_the_steps(m):
    """Back to back (kernels starting early on one another) as with a wait after every call."""
    need_gpu()
    w, t = weights(1), tokens(m, m)
    for _ in range(20):
        got = layer(w, t)
    q, s, res, y = qk.add_rmsnorm_quant_per_token(t["x"], w["norm1"], t["res"], want_norm=True)
    torch.cuda.synchronize()
    h = qk.w8a8_lora_gemm(q, w["w"], s, w["sw"], y, w["la"], w["lb"], t["ids"])
    torch.cuda.synchronize()
    q, s, res, _ = qk.add_rmsnorm_quant_per_token(h, w["norm2"], res)
    torch.cuda.synchronize()
    out = qk.w8a8_moe_layer(q, s, t["top"], t["wt"], w["w13"], w["s13"], w["w2"], w["s2"])
    torch.cuda.synchronize()
    assert same(got, (out, res))
    assert bool(out.isfinite().all()) and float(out.float().abs().max()) > 0
    assert qk.device_status() == qk.QK_OK


@pytest.mark.parametrize("m", [3, 33])
def test_chain_captured(m):
    """A captured layer replayed on new inputs, and two of them replayed on two streams at once."""
    need_gpu()
    w = weights(2)
    graphs, buffers, outs = [], [], []
    for k in range(2):
        t = tokens(m, 100 + k)
        layer(w, t)  # (first use outside the capture)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(w, t))
        graphs.append(g)
        buffers.append(t)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(8):
        fresh = [tokens(m, 10 * turn + k) for k in range(2)]
        want = [layer(w, f) for f in fresh]
        for k in range(2):
            for name, v in fresh[k].items():
                buffers[k][name].copy_(v)
        torch.cuda.synchronize()
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                for _ in range(3):
                    graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert same(outs[k], want[k])
    del graphs


@pytest.mark.parametrize("m", [4, 130])
def test_on_another_stream(m):
    """stream=: what the call allocates belongs to that stream, so nothing is handed out before it ran."""
    need_gpu()
    w, t = weights(3), tokens(m, 7)
    t["res"] = t["res"].clone()
    a, sa = qk.quantize_per_token(t["x"])
    want = qk.w8a8_lora_gemm(a, w["w"], sa, w["sw"], t["x"], w["la"], w["lb"], t["ids"])
    full = layer(w, t) if m <= 64 else None
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(30):
        got.append(qk.w8a8_lora_gemm(a, w["w"], sa, w["sw"], t["x"], w["la"], w["lb"], t["ids"], stream=side))
        # memory of the current stream, written at once: a workspace taken from it would be overwritten
        torch.empty(4 << 20, dtype=torch.uint8, device="cuda").fill_(255)
        if full is not None:
            assert len(layer(w, t, stream=side)) == 2
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    if full is not None:
        again = layer(w, t, stream=side)
        side.synchronize()
        assert same(again, full)


def test_one_workspace_for_calls_of_all_kinds():
    """A workspace used again by the next call on the stream, while the last one's kernels still run: tokens
    without any expert or adapter (kernels with nothing to do end at once) between ordinary ones."""
    need_gpu()
    w = weights(8)
    kinds = []
    for k, m in enumerate((6, 64, 1, 17)):
        t = tokens(m, 60 + k)
        a, sa = qk.quantize_per_token(t["x"])
        for none in (False, True):
            top = torch.full_like(t["top"], -1) if none else t["top"]
            ids = torch.full_like(t["ids"], -1) if none else t["ids"]
            kinds.append((lambda ws, a=a, sa=sa, top=top, t=t: qk.w8a8_moe_layer(
                a, sa, top, t["wt"], w["w13"], w["s13"], w["w2"], w["s2"], workspace=ws),
                lambda ws, a=a, sa=sa, ids=ids, t=t: qk.w8a8_lora_gemm(
                    a, w["w"], sa, w["sw"], t["x"], w["la"], w["lb"], ids, workspace=ws)))
    big = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    want = []
    for pair in kinds:
        for call in pair:
            want.append(call(None))
            torch.cuda.synchronize()
    for _ in range(10):
        big.fill_(255)
        got = [call(big) for pair in kinds for call in pair]
        assert same(got, want)


def test_one_workspace_for_long_batches():
    """Batches of different lengths, orders of adapters and numbers of groups, one behind another: each writes its
    groups and sums where the last one's kernels have just read theirs."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(9)
    n, k, rank, adapters = 1032, 528, 24, 7
    b = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand(n, generator=g, device="cuda") / 1000
    la = (torch.randn((adapters, rank, k), generator=g, device="cuda") / 20).bfloat16()
    lb = torch.randn((adapters, n, rank), generator=g, device="cuda").bfloat16()
    ws = torch.full((32 << 20,), 255, dtype=torch.uint8, device="cuda")
    calls = []
    for m in (70, 1024, 2500, 65, 1300):
        x = torch.randn((m, k), generator=g, device="cuda").bfloat16()
        a, sa = qk.quantize_per_token(x)
        ids = torch.randint(-1, adapters, (m,), generator=g, device="cuda", dtype=torch.int32)
        for order in (ids, torch.sort(ids, descending=True).values, torch.full_like(ids, -1), torch.full_like(ids, 3)):
            calls.append(lambda ws, a=a, sa=sa, x=x, order=order: qk.w8a8_lora_gemm(
                a, b, sa, sw, x, la, lb, order, workspace=ws))
    want = []
    for call in calls:
        want.append(call(None))
        torch.cuda.synchronize()
    for _ in range(5):
        got = [call(ws) for call in calls]
        got += [call(ws) for call in reversed(calls)]
        assert same(got, want + want[::-1])


def test_projection_captured_with_split_k():
    """The GEMM's own workspace has to be cleared in the replay too."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(3)
    m, n, k = 300, 2304, 512
    x = torch.randn((m, k), generator=g, device="cuda").bfloat16()
    b = torch.randint(-127, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand(n, generator=g, device="cuda") / 1000
    la = (torch.randn((2, 8, k), generator=g, device="cuda") / 20).bfloat16()
    lb = torch.randn((2, n, 8), generator=g, device="cuda").bfloat16()
    ids = torch.randint(-1, 2, (m,), generator=g, device="cuda", dtype=torch.int32)
    a, sa = qk.quantize_per_token(x)
    want = qk.w8a8_lora_gemm(a, b, sa, sw, x, la, lb, ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = qk.w8a8_lora_gemm(a, b, sa, sw, x, la, lb, ids)
    for _ in range(5):
        out.zero_()
        graph.replay()
        graph.replay()
        assert torch.equal(out, want)
    del graph


def test_from_several_threads():
    """Calls of several threads on one stream and on their own: each has its own workspace."""
    need_gpu()
    w = weights(4)
    inputs = [tokens(3 + k, 50 + k) for k in range(4)]
    want = [layer(w, t) for t in inputs]
    torch.cuda.synchronize()
    bad = []

    def work(k, own):
        try:
            stream = torch.cuda.Stream() if own else torch.cuda.default_stream()
            with torch.cuda.stream(stream):
                for _ in range(25):
                    got = layer(w, inputs[k])
                    stream.synchronize()
                    if not same(got, want[k]):
                        bad.append(k)
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    for own in (False, True):
        threads = [threading.Thread(target=work, args=(k, own)) for k in range(4)]
        for th in threads:
            th.start()
        for th in threads:
            th.join()
    assert not bad


def test_another_device_is_current():
    need_gpu()
    if torch.cuda.device_count() < 2:
        pytest.skip("one device")
    w, t = weights(5, "cuda:1"), tokens(4, 1, "cuda:1")
    got = layer(w, t)
    with torch.cuda.device(1):
        assert same(got, layer(w, t))


def test_stream_of_another_device_and_mixed_devices_are_refused():
    need_gpu()
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        qk.add_rmsnorm_quant_per_token(x, torch.ones(64, dtype=torch.bfloat16))
    if torch.cuda.device_count() > 1:
        with pytest.raises(ValueError):
            qk.add_rmsnorm_quant_per_token(x, x[0], stream=torch.cuda.Stream(device=1))


def test_weights_written_just_before():
    """A kernel that lets its dependents start early may have written anything but the weights just before: here
    torch writes every input, the weights too, between calls on one stream."""
    need_gpu()
    w, t = weights(6), tokens(6, 2)
    other_w, other_t = weights(7), tokens(6, 3)
    want = layer(w, t), layer(other_w, other_t)
    live_w = {n: v.clone() for n, v in w.items()}
    live_t = {n: v.clone() for n, v in t.items()}
    for turn in range(10):
        k = turn % 2
        for n, v in (w, other_w)[k].items():
            live_w[n].copy_(v)
        for n, v in (t, other_t)[k].items():
            live_t[n].copy_(v)
        assert same(layer(live_w, live_t), want[k])
