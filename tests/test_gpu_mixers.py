"""The operators between a layer's projections run together: a DecayLayer against its 64-bit form, an attention
layer that turns its queries and keys itself, and a hybrid period of all of them, captured."""
import pytest
import torch

import mixer_ref as mr
import paged_ref as ref
from gated_deltanet_linear_09_gb300 import hybrid, runtime, synth

pytestmark = pytest.mark.gpu


def bf16(x):
    return x.to(torch.bfloat16).double()


def ints(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def batch_of(new, lens, table):
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    return runtime.KVBatch(ints(cu), ints(lens), table, cu[-1], max(new))


@pytest.mark.parametrize("Hk,Hv,dk,dv", [(2, 4, 64, 64), (1, 2, 128, 128)])
def test_decay_layer(Hk, Hv, dk, dv):
    """Prompts in two pieces, then single tokens, against whole sequences.  Each stored value is rounded to bf16
    (2^-8 at most, a step where an f32 sum falls on the other side); the attention rounds scores and states:
    2^-5 of a row's length holds a few of these one after another (a head's norm divides by its length, which
    may be a fraction of its terms')."""
    hidden, lens, n = 128, [150, 37, 5], 3
    w = hybrid.decay_weights(hidden, Hk, Hv, dk, dv, 3)
    plan = runtime.Rotary(dk, base=1e4)
    layer = hybrid.DecayLayer(runtime.DecayAttention(Hk, Hv, dk, dv, n + 1), w, rotary=plan)
    g = torch.Generator().manual_seed(5)
    xs = [torch.randn((t, hidden), generator=g).to(torch.bfloat16) for t in lens]
    w = {k: v.cpu().double() for k, v in w.items()}
    want = []
    for x in xs:
        T, x = x.shape[0], x.double()
        q, k = (bf16(x @ w[m].T).view(T, Hk, dk) for m in ("w_q", "w_k"))
        q, k = (bf16(mr.rotated(t, range(T), plan.frequencies)) for t in (q, k))
        v, z = (bf16(x @ w[m].T).view(T, Hv, dv) for m in ("w_v", "w_z"))
        o, _, _, _ = mr.decay(torch.zeros(Hv, dk, dv, dtype=torch.float64), q, k, v, w["log_decay"])
        y, _ = mr.block(bf16(o).reshape(T, -1), post=w["norm"], gate=z.reshape(T, -1), gate_act="silu", offset=1.0)
        want.append(bf16(y) @ w["w_out"].T)
    got, done, slots = [[] for _ in lens], [0] * n, ints([2, 0, 3])
    for new in ([100, 20, 1], [48, 15, 2], [1, 1, 1], [1, 1, 1]):
        x = torch.cat([xs[i][d:d + m] for i, (d, m) in enumerate(zip(done, new))]).cuda()
        pos = ints([d + j for d, m in zip(done, new) for j in range(m)])
        if max(new) == 1:
            y = layer.forward(x, slots, positions=pos)
        else:
            init = torch.tensor([d > 0 for d in done], dtype=torch.uint8, device="cuda")
            y = layer.forward(x, slots, ints([sum(new[:i]) for i in range(n + 1)]), init, positions=pos)
        done = [d + m for d, m in zip(done, new)]
        for i, part in enumerate(y.cpu().double().split(new)):
            got[i].append(part)
    assert done == lens and int(layer.status.item()) == 0 and int(layer.attention.status.item()) == 0
    for a, b in zip(got, want):
        diff = (torch.cat(a) - b).norm(dim=-1) / b.norm(dim=-1)
        assert (diff <= 2.0 ** -5).all(), float(diff.max())
    with pytest.raises(ValueError):
        layer.forward(xs[0].cuda(), slots)


@pytest.mark.parametrize("quantised", [False, True])
def test_attention_layer_turns_its_keys(quantised):
    """With a rotation of its own: the norms, rotation and append of one launch against the separate calls (which
    round to bf16 in between: half a step, 2^-8, of q and k each, twice 2^-8 of the outputs' length with
    what the scores make of it, 2^-5 with an 8-bit cache's other roundings)."""
    hidden, Hq, H, D = 128, 4, 2, 128
    w = hybrid.attention_weights(hidden, Hq, H, D, 6)
    plan = runtime.Rotary(64, base=1e4)
    new, table = [40, 7, 1], torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3)
    pos = ints([j for m in new for j in range(m)])
    x = torch.randn((48, hidden), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    outs = []
    for own in (True, False):
        cache = runtime.PagedKVCache(9, 16, H, D, quantised)
        layer = hybrid.AttentionLayer(cache, Hq, w, rotary=plan if own else None)
        b = batch_of(new, new, table)
        outs.append(layer.forward(b, x, None if own else lambda q, k: plan.apply(pos, q, k)).double())
        assert int(cache.status.item()) == 0
        if own:
            with pytest.raises(ValueError):
                layer.forward(b, x, lambda q, k: (q, k))
    diff = (outs[0] - outs[1]).norm(dim=-1) / outs[1].norm(dim=-1)
    assert bool((diff <= 2.0 ** (-4 if quantised else -5)).all()), float(diff.max())


def test_period_in_a_graph():
    """A period of Gated DeltaNet, decayed and attention layers with norms after them: eager decoding steps and the
    replayed graph of one give the same bits."""
    geo, hidden, n = synth.Geometry(2, 4, 64, 64), 256, 3

    def run(graphed):
        cache = runtime.PagedKVCache(3 * n, 16, 2, 64, True)
        period = hybrid.make_period(geo, hidden, cache, 4, n, linear=3, seed=7, decayed=2, rotary=runtime.Rotary(32), post_norms=True,
                                    residual_scale=0.5)
        table = torch.arange(3 * n, dtype=torch.int32, device="cuda").view(n, 3)
        g = torch.Generator(device="cuda").manual_seed(8)
        slots, new = torch.arange(n, dtype=torch.int32, device="cuda"), [20, 3, 11]
        b = batch_of(new, new, table)
        x = torch.randn((sum(new), hidden), generator=g, device="cuda").to(torch.bfloat16)
        y, total = period.step(b, x, slots, b.tensors[0], torch.zeros(n, dtype=torch.uint8, device="cuda"),
                               positions=ints([j for m in new for j in range(m)]))
        assert y.isfinite().all() and total.isfinite().all()
        b = batch_of([1] * n, new, table)
        x = torch.randn((n, hidden), generator=g, device="cuda").to(torch.bfloat16)
        places, outs = torch.empty_like(b.tensors[1]), []

        def step():
            places.copy_(b.tensors[1])
            b.tensors[1].add_(1)
            return period.step(b, x, slots, positions=places)
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
        assert int(cache.status.item()) == 0
        return outs
    for a, b in zip(run(False), run(True)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_example_runs_with_them(capsys):
    assert hybrid.main(["--sequences", "3", "--prompt", "150", "--piece", "64", "--steps", "4", "--rotary", "--decayed", "2",
                        "--post-norms"]) == 0
    assert "decode: 3 sequences" in capsys.readouterr().out


def test_append_rotated_on_a_late_stream():
    """What a call on another stream allocates and writes is that stream's."""
    case = ref.Case([3, 1], [200, 90], 2, 64, 16, False, seed=61)
    plan = runtime.Rotary(64)
    q, k, v = (torch.randn((4, h, 64), device="cuda").to(torch.bfloat16) for h in (4, 2, 2))
    cache, b = case.filled_cache(runtime), case.device_batch(runtime)
    want = cache.append_rotated(b, plan, q, k, v)
    pages = cache.k_pages.clone()
    late = torch.cuda.Stream()
    late.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(late):
        torch.cuda._sleep(20_000_000)
    got = cache.append_rotated(b, plan, q, k, v, stream=late)
    with torch.cuda.stream(late):
        kept = got.clone()
    del got
    for _ in range(4):
        torch.full((4, 4, 64), 7, dtype=torch.bfloat16, device="cuda")
    late.synchronize()
    assert torch.equal(kept, want) and torch.equal(cache.k_pages.view(torch.int16), pages.view(torch.int16))
