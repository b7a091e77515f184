"""The norm, cache and attention operators run together: the gated attention layer against its
64-bit form, a hybrid period, its captured decoding step, and calls on two streams."""
import pytest
import torch

import paged_ref as ref
from gated_deltanet_linear_09_gb300 import hybrid, runtime, synth

pytestmark = pytest.mark.gpu


def bf16(x):
    return x.to(torch.bfloat16).double()


def norm64(x, w, eps=1e-6):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (1.0 + w)


def layer64(xs, w, Hq, H, D):
    """An attention layer over whole sequences in 64 bits, rounded to bf16 where the layer stores
    bf16."""
    outs = []
    for x in xs:
        T = x.shape[0]
        x = x.double()
        qg = bf16(x @ w["w_q"].double().T).view(T, Hq, 2 * D)
        gate = torch.sigmoid(qg[..., D:])
        k = bf16(norm64(bf16(x @ w["w_k"].double().T).view(T, H, D), w["k_norm"].double()))
        v = bf16(x @ w["w_v"].double().T).view(T, H, D)
        q = bf16(norm64(qg[..., :D], w["q_norm"].double()))
        kq, vq = (t.repeat_interleave(Hq // H, 1) for t in (k, v))
        seen = torch.tril(torch.ones(T, T, dtype=torch.bool))
        s = torch.einsum("thd,jhd->htj", q, kq) / D ** 0.5
        p = torch.softmax(s.masked_fill(~seen, -torch.inf), -1)
        o = torch.einsum("htj,jhd->thd", p, vq) * gate
        outs.append(bf16(o).reshape(T, Hq * D) @ w["w_out"].double().T)
    return outs


def batch_of(new, lens, table):
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    t = [torch.tensor(a, dtype=torch.int32, device="cuda") for a in (cu, lens)]
    return runtime.KVBatch(t[0], t[1], table, cu[-1], max(new))


@pytest.mark.parametrize("Hq,H,D", [(4, 2, 64), (8, 1, 128), (2, 2, 256)])
def test_attention_layer(Hq, H, D):
    """Prompts in two pieces, then tokens one at a time, against the whole sequences.  The layer
    rounds the probabilities, the attention's output and the projection's by half a bf16 step (2^-8)
    each; where an f32 sum falls on the other side of a rounding than the 64-bit one, a stored value
    is a step (2^-7) off, which few are: 2^-6 of a row's length holds all of it."""
    hidden, lens, n = 128, [70, 37, 5], 3
    w = hybrid.attention_weights(hidden, Hq, H, D, 3)
    cache = runtime.PagedKVCache(n * 5, 16, H, D)
    table = torch.randperm(n * 5, generator=torch.Generator().manual_seed(4)).to(torch.int32).view(n, 5).cuda()
    layer = hybrid.AttentionLayer(cache, Hq, w)
    g = torch.Generator().manual_seed(5)
    xs = [torch.randn((t, hidden), generator=g).to(torch.bfloat16) for t in lens]
    want = layer64(xs, {k: v.cpu() for k, v in w.items()}, Hq, H, D)
    got, done = [[] for _ in lens], [0] * n
    for new in ([40, 20, 1], [28, 15, 2], [1, 1, 1], [1, 1, 1]):
        x = torch.cat([xs[i][d:d + m] for i, (d, m) in enumerate(zip(done, new))]).cuda()
        done = [d + m for d, m in zip(done, new)]
        y = layer.forward(batch_of(new, done, table), x).cpu().double()
        for i, part in enumerate(y.split(new)):
            got[i].append(part)
    assert done == lens and int(cache.status.item()) == 0 and int(layer.status.item()) == 0
    for a, b in zip(got, want):
        diff = (torch.cat(a) - b).norm(dim=-1) / b.norm(dim=-1)
        assert (diff <= 2.0 ** -6).all(), float(diff.max())


def test_rotation_is_applied():
    """The keys that the cache holds are the rotated ones."""
    w = hybrid.attention_weights(64, 2, 1, 64, 6)
    cache = runtime.PagedKVCache(2, 16, 1, 64)
    layer = hybrid.AttentionLayer(cache, 2, w)
    b = batch_of([5], [5], torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
    x = torch.randn((5, 64), device="cuda").to(torch.bfloat16)
    seen = {}

    def rotate(q, k):
        seen["k"] = k * 2
        return q, seen["k"]
    layer.forward(b, x, rotate)
    assert torch.equal(cache.read(b)[0], seen["k"])


@pytest.mark.parametrize("quantised", [False, True])
def test_period_in_a_graph(quantised):
    """Eager decoding steps and the replayed graph of one give the same bits."""
    geo, hidden, n = synth.Geometry(2, 4, 64, 64), 256, 3

    def run(graphed):
        cache = runtime.PagedKVCache(3 * n, 16, 2, 64, quantised)
        period = hybrid.make_period(geo, hidden, cache, 4, n, linear=2, seed=7)
        table = torch.arange(3 * n, dtype=torch.int32, device="cuda").view(n, 3)
        g = torch.Generator(device="cuda").manual_seed(8)
        slots = torch.arange(n, dtype=torch.int32, device="cuda")
        new = [20, 3, 11]
        b = batch_of(new, new, table)
        x = torch.randn((sum(new), hidden), generator=g, device="cuda").to(torch.bfloat16)
        y, total = period.step(b, x, slots, b.tensors[0], torch.zeros(n, dtype=torch.uint8, device="cuda"))
        assert y.isfinite().all() and total.isfinite().all()
        b = batch_of([1] * n, new, table)
        x = torch.randn((n, hidden), generator=g, device="cuda").to(torch.bfloat16)
        outs = []

        def step():
            b.tensors[1].add_(1)
            return period.step(b, x, slots)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            outs.append([t.clone() for t in step()])
            side.synchronize()
            graph = torch.cuda.CUDAGraph()
            if graphed:
                with torch.cuda.graph(graph, stream=side):
                    y = step()
            for _ in range(4):
                if graphed:
                    graph.replay()
                else:
                    y = step()
                outs.append([t.clone() for t in y])
            side.synchronize()
        assert int(cache.status.item()) == 0 and int(period.attention.status.item()) == 0
        return outs
    for a, b in zip(run(False), run(True)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_have_their_own_workspace():
    """Attention over one cache on two streams at once: each gives what it gives alone."""
    case = ref.Case([1] * 6, [900, 3000, 17, 2500, 1, 1200], 2, 128, 32, False, seed=9)
    cache = case.filled_cache(runtime)
    b = case.device_batch(runtime)
    q = [torch.randn((6, 8, 128), device="cuda").to(torch.bfloat16) for _ in range(2)]
    want = [cache.attend(b, x).clone() for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = [torch.empty_like(x) for x in q]
    torch.cuda.synchronize()
    assert cache.workspace(8, streams[0]).data_ptr() != cache.workspace(8, streams[1]).data_ptr()
    assert cache.workspace(8, streams[0]).data_ptr() == cache.workspace(8, streams[0]).data_ptr()
    for _ in range(20):
        for s, x, o in zip(streams, q, out):
            cache.attend(b, x, out=o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_example_runs(capsys):
    assert hybrid.main(["--sequences", "3", "--prompt", "150", "--piece", "64", "--steps", "4"]) == 0
    assert "decode: 3 sequences" in capsys.readouterr().out
