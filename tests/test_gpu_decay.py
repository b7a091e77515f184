"""Linear attention with a decay for each head, single tokens and whole prompts, against the recurrence in 64
bits.

Tolerances.  size = scale sum |q||S| and M = sum e^(..)|k||v| are what the roundings act on.  Step: f32 sums of
at most dk terms and T updates, 2^-24 each: 2^-16 size (2^-16 M) holds 2^8 of them; the output's half step.
Prompt: scores times their decays, and the states, are rounded to bf16 for the output (2^-9 of each, at most 2^-8
size together, as only one of the two holds any term), in f32 sums; the state is summed from keys exact to
2^-16 of each, in f32 sums over chunks: 2^-14 M.  Decays of f32 logarithms: 2^-23 of each sum of up to 128 of them."""
import math

import pytest
import torch

import mixer_ref as mr
from gated_deltanet_linear_09_gb300 import gdn, runtime

pytestmark = pytest.mark.gpu


def inputs(lead, Hk, Hv, dk, dv, seed, gated, rate=1.0):
    g = torch.Generator().manual_seed(seed)
    row = torch.randn((*lead, 2 * Hk * dk + Hv * dv), generator=g).to(torch.bfloat16)
    if gated:
        decay = -rate * torch.rand((*lead, Hv), generator=g)
    else:
        decay = -rate * 2.0 ** (-8.0 * torch.arange(1, Hv + 1) / Hv)
    return row, decay


def views(row, Hk, Hv, dk, dv):
    q = row[..., :Hk * dk].unflatten(-1, (Hk, dk))
    k = row[..., Hk * dk:2 * Hk * dk].unflatten(-1, (Hk, dk))
    return q, k, row[..., 2 * Hk * dk:].unflatten(-1, (Hv, dv))


def pool(slots, Hv, dk, dv, seed):
    return torch.randn((slots, Hv, dk, dv), generator=torch.Generator().manual_seed(seed))


def out_bound(want, size, rel):
    return rel * size + mr.BF16 * (want.abs() + rel * size) + 1e-37


DIMS = [(128, 128), (64, 64), (64, 128), (128, 64)]


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("T,gated", [(1, False), (1, True), (3, True), (8, False)])
def test_step(dk, dv, T, gated):
    for rows, Hk, Hv in ((1, 1, 1), (5, 2, 6), (33, 4, 4)):
        state = pool(rows + 2, Hv, dk, dv, 1)
        row, decay = inputs((rows, T), Hk, Hv, dk, dv, rows, gated)
        slots = torch.randperm(rows + 2, generator=torch.Generator().manual_seed(2))[:rows].to(torch.int32)
        if rows > 1:
            slots[1] = -1
        layer = runtime.DecayAttention.over(state.cuda(), Hk)
        q, k, v = views(row.cuda(), Hk, Hv, dk, dv)
        if T == 1:
            q, k, v = (x[:, 0] for x in (q, k, v))
            got = layer.step(slots.cuda(), q, k, v, (decay[:, 0] if gated else decay).contiguous().cuda())[:, None]
        else:
            got = layer.step(slots.cuda(), q, k, v, decay.cuda())
        left = state.clone()
        q, k, v = views(row, Hk, Hv, dk, dv)
        for i, s in enumerate(slots.tolist()):
            if s < 0:
                assert bool((got[i] == 0).all())
                continue
            o, S, size, M = mr.decay(state[s].double(), *(x[i].double() for x in (q, k, v)),
                                     (decay[i] if gated else decay).double())
            mr.close(got[i], o, out_bound(o, size, 2.0 ** -16))
            mr.close(layer.state[s], S, 2.0 ** -16 * M)
            left[s] = layer.state[s].cpu()
        assert torch.equal(layer.state.cpu(), left) and int(layer.status.item()) == 0


def run_prompts(lens, Hk, Hv, dk, dv, gated, init, seed=3, rate=1.0, scale=0.0, slots=None, row=None, decay=None, state=None):
    """(outputs, layer, checked): the call, and the check against the recurrence."""
    n, total = len(lens), sum(lens)
    if state is None:
        state = pool(n + 1, Hv, dk, dv, seed)
    if row is None:
        row, decay = inputs((total,), Hk, Hv, dk, dv, seed, gated, rate)
    cu = [sum(lens[:i]) for i in range(n + 1)]
    if slots is None:
        slots = torch.randperm(state.shape[0], generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32)
    layer = runtime.DecayAttention.over(state.cuda(), Hk, scale)
    q, k, v = views(row.cuda(), Hk, Hv, dk, dv)
    flags = None if init is None else torch.tensor(init, dtype=torch.uint8, device="cuda")
    got = layer.prefill(torch.tensor(cu, dtype=torch.int32, device="cuda"), slots.cuda(), flags, q, k, v, decay.cuda())
    q, k, v = views(row, Hk, Hv, dk, dv)
    left = state.clone()
    for i, s in enumerate(slots.tolist()):
        part = slice(cu[i], cu[i + 1])
        if s < 0:
            assert bool((got[part] == 0).all())
            continue
        S0 = state[s].double() if init is not None and init[i] else torch.zeros(Hv, dk, dv, dtype=torch.float64)
        o, S, size, M = mr.decay(S0, *(x[part].double() for x in (q, k, v)),
                                 (decay[part] if decay.dim() > 1 else decay).double(), scale or None)
        mr.close(got[part], o, out_bound(o, size, 2.0 ** -8 + 2.0 ** -12), f"sequence {i}")
        mr.close(layer.state[s], S, 2.0 ** -14 * M, f"state of sequence {i}")
        left[s] = layer.state[s].cpu()
    assert torch.equal(layer.state.cpu(), left)
    return got, layer


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("gated", [False, True])
def test_prompts(dk, dv, gated):
    lens = [1, 0, 127, 128, 129, 5, 300, 64, 65]
    _, layer = run_prompts(lens, 2, 4, dk, dv, gated, [i % 2 for i in range(len(lens))])
    assert int(layer.status.item()) == 0


@pytest.mark.parametrize("lens,Hk,Hv", [([1], 1, 1), ([2500], 1, 2), ([700, 1, 1500], 3, 3), ([1] * 40, 1, 3), ([128] * 3, 1, 4)])
def test_lengths(lens, Hk, Hv):
    """Long sequences (several pieces each), many short ones, whole chunks; fresh and continued."""
    run_prompts(lens, Hk, Hv, 128, 128, True, None)
    run_prompts(lens, Hk, Hv, 128, 128, False, [1] * len(lens), rate=0.05)


def test_decays_of_any_size():
    """Hardly any decay, strong ones, tokens that empty the state, a growing state; a given scale."""
    T, Hv = 400, 5
    row, _ = inputs((T,), 1, Hv, 128, 128, 9, True)
    g = torch.Generator().manual_seed(10)
    decay = torch.empty(T, Hv)
    decay[:, 0] = 0.0
    decay[:, 1] = -20.0 * torch.rand(T, generator=g)
    decay[:, 2] = -0.01
    decay[torch.tensor([0, 3, 127, 128, 200, 399]), 2] = -math.inf
    decay[:, 3] = 0.01
    decay[:, 4] = torch.where(torch.rand(T, generator=g) < 0.1, -300.0, -0.1)
    run_prompts([T], 1, Hv, 128, 128, True, [1], row=row, decay=decay, scale=0.5)


def test_prompt_then_steps_is_one_prompt():
    """A prompt in two calls and single tokens after it leave the state of one call, to the roundings."""
    Hk, Hv, d, T = 2, 4, 128, 333
    row, decay = inputs((T,), Hk, Hv, d, d, 20, True)
    q, k, v = views(row.cuda(), Hk, Hv, d, d)
    g = decay.cuda()
    one = torch.zeros(1, dtype=torch.int32, device="cuda")

    def cu(n):
        return torch.tensor([0, n], dtype=torch.int32, device="cuda")
    a = runtime.DecayAttention(Hk, Hv, d, d, 1)
    whole = a.prefill(cu(T), one, None, q, k, v, g)
    b = runtime.DecayAttention(Hk, Hv, d, d, 1)
    parts = [b.prefill(cu(200), one, None, q[:200], k[:200], v[:200], g[:200]),
             b.prefill(cu(130), one, torch.ones(1, dtype=torch.uint8, device="cuda"), q[200:330], k[200:330], v[200:330], g[200:330])]
    for t in range(330, T):
        parts.append(b.step(one, q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1]))
    o, S, size, M = mr.decay(torch.zeros(Hv, d, d, dtype=torch.float64), *(x.cpu().double() for x in (q, k, v)), decay.double())
    for got, layer in ((whole, a), (torch.cat(parts), b)):
        mr.close(got, o, out_bound(o, size, 2.0 ** -8 + 2.0 ** -12))
        mr.close(layer.state[0], S, 2.0 ** -14 * M)


def test_bad_slots_and_lengths():
    """Slots out of range and padding: zeros, no state touched; an inconsistent cu_seqlens: nothing but zeros."""
    lens = [140, 20, 30]
    slots = torch.tensor([1, -1, 0], dtype=torch.int32)
    _, layer = run_prompts(lens, 1, 2, 64, 64, True, None, slots=slots)
    assert int(layer.status.item()) == 0
    row, decay = inputs((190,), 1, 2, 64, 64, 5, True)
    q, k, v = views(row.cuda(), 1, 2, 64, 64)
    for cu, idx, want in (([0, 140, 160, 190], [1, 9, 0], gdn.GDN_STATUS_SLOT_RANGE), ([0, 160, 140, 190], [0, 1, 2], gdn.GDN_STATUS_BAD_SEQLENS),
                          ([0, 10, 20, 191], [0, 1, 2], gdn.GDN_STATUS_BAD_SEQLENS), ([-5, 10, 20, 190], [0, 1, 2], gdn.GDN_STATUS_BAD_SEQLENS),
                          ([0, 10, 20, 150], [0, 1, 2], 0), ([7, 10, 20, 190], [0, 1, 2], gdn.GDN_STATUS_BAD_SEQLENS)):
        state = pool(3, 2, 64, 64, 4)
        layer = runtime.DecayAttention.over(state.cuda(), 1)
        out = torch.full((190, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        layer.prefill(torch.tensor(cu, dtype=torch.int32, device="cuda"), torch.tensor(idx, dtype=torch.int32, device="cuda"), None,
                      q, k, v, decay.cuda(), out=out)
        assert int(layer.status.item()) == want, cu
        if want == gdn.GDN_STATUS_BAD_SEQLENS:
            assert bool((out == 0).all()) and torch.equal(layer.state.cpu(), state)
        elif want:
            assert bool((out[140:160] == 0).all()) and torch.equal(layer.state[2].cpu(), state[2])
            assert not torch.equal(layer.state[1].cpu(), state[1])
        else:
            assert bool((out[150:] == 0).all())                      # tokens of no sequence
    layer = runtime.DecayAttention.over(pool(3, 2, 64, 64, 4).cuda(), 1)
    out = layer.step(torch.tensor([0, 3], dtype=torch.int32, device="cuda"), q[:2], k[:2], v[:2], decay[:2].cuda())
    assert int(layer.status.item()) == gdn.GDN_STATUS_SLOT_RANGE and bool((out[1] == 0).all())


def test_later_tokens_have_no_influence():
    """A NaN or an infinity in a later token's value or key leaves the earlier outputs' bits alone, and other
    heads and sequences altogether; the tokens from it on, and the state, have it."""
    lens, Hk, Hv, d = [300, 200], 1, 2, 128
    row, decay = inputs((500,), Hk, Hv, d, d, 30, True, rate=0.01)
    want, clean = run_prompts(lens, Hk, Hv, d, d, True, None, row=row, decay=decay)
    for t, at, value in ((150, 2 * d + 5, math.nan), (255, 2 * d + d + 7, math.inf), (299, 2 * d, -math.inf), (140, d + 3, math.nan)):
        spoiled = row.clone()
        spoiled[t, at] = value
        layer = runtime.DecayAttention.over(pool(3, Hv, d, d, 3).cuda(), Hk)
        q, k, v = views(spoiled.cuda(), Hk, Hv, d, d)
        cu = torch.tensor([0, 300, 500], dtype=torch.int32, device="cuda")
        slots = torch.randperm(3, generator=torch.Generator().manual_seed(3))[:2].to(torch.int32)
        got = layer.prefill(cu, slots.cuda(), None, q, k, v, decay.cuda())
        assert torch.equal(got[:t], want[:t]) and torch.equal(got[300:], want[300:])
        s = int(slots[0])
        if at >= 2 * d:                                              # one column of one head
            h, c = divmod(at - 2 * d, d)
            assert not bool(got[t:300, h, c].isfinite().any())
            others = torch.ones(Hv, d, dtype=torch.bool)
            others[h, c] = False
            assert torch.equal(got[:, others.cuda()], want[:, others.cuda()])
            assert not bool(layer.state[s, h, :, c].isfinite().any())
            assert torch.equal(layer.state[s][:, :, :][others[:, None, :].expand(Hv, d, d).cuda()],
                               clean.state[s][others[:, None, :].expand(Hv, d, d).cuda()])
        else:
            assert bool(got[t:300].isnan().all()) and bool(layer.state[s, :, at - d].isnan().all())


def test_graphs_streams_and_repeats():
    """The same bits on another stream, in a graph, and again; two graphs replayed beside each other."""
    lens, Hk, Hv, d = [900, 100, 1], 1, 3, 128
    row, decay = inputs((1001,), Hk, Hv, d, d, 40, True)
    want, _ = run_prompts(lens, Hk, Hv, d, d, True, None, row=row, decay=decay)
    q, k, v = views(row.cuda(), Hk, Hv, d, d)
    g = decay.cuda()
    cu = torch.tensor([0, 900, 1000, 1001], dtype=torch.int32, device="cuda")
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    layers = [runtime.DecayAttention(Hk, Hv, d, d, 3) for _ in range(2)]
    outs = [torch.zeros_like(want) for _ in layers]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    layers[0].prefill(cu, slots, None, q, k, v, g, out=outs[0], stream=side)
    side.synchronize()
    assert torch.equal(outs[0], want)
    graphs = []
    for layer, o in zip(layers, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for _ in range(3):
                layer.prefill(cu, slots, None, q, k, v, g, out=o)
        graphs.append(graph)
        o.zero_()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert torch.equal(layers[0].state, layers[1].state)


def test_many_sequences():
    """More sequences than a CTA has threads, most of them short, some empty; and ranges that do not fit together
    among many, such as lengths that wrap around 32 bits."""
    g = torch.Generator().manual_seed(50)
    lens = torch.randint(0, 5, (1500,), generator=g).tolist()
    lens[700], lens[1499] = 400, 150
    run_prompts(lens, 1, 1, 64, 64, True, [i % 3 == 0 for i in range(1500)])
    row, decay = inputs((100,), 1, 2, 64, 64, 5, True)
    q, k, v = views(row.cuda(), 1, 2, 64, 64)
    for at, cuts in ((20, [2 ** 31 - 1, -2 ** 31, -1]), (0, [3]), (30, [101, 100]), (39, [50, 20])):
        cu = [0] * at + cuts + [100] * (41 - at - len(cuts))
        state = pool(40, 2, 64, 64, 4)
        layer = runtime.DecayAttention.over(state.cuda(), 1)
        out = layer.prefill(torch.tensor(cu, dtype=torch.int32, device="cuda"), torch.arange(40, dtype=torch.int32, device="cuda"), None,
                            q, k, v, decay.cuda())
        assert int(layer.status.item()) == gdn.GDN_STATUS_BAD_SEQLENS, cuts
        assert bool((out == 0).all()) and torch.equal(layer.state.cpu(), state)


def test_no_tokens():
    """Sequences without any tokens: states begin, or stay."""
    state = pool(4, 2, 128, 64, 6)
    for n in (3, 40):
        layer = runtime.DecayAttention.over(state.cuda(), 1)
        slots = torch.full((n,), -1, dtype=torch.int32)
        slots[:3] = torch.tensor([2, 0, -1])
        flags = torch.zeros(n, dtype=torch.uint8, device="cuda")
        flags[0] = 1
        nothing = torch.zeros((0, 2, 128), dtype=torch.bfloat16, device="cuda")
        out = layer.prefill(torch.zeros(n + 1, dtype=torch.int32, device="cuda"), slots.cuda(), flags, nothing[:, :1], nothing[:, :1],
                            torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros(2, device="cuda"))
        want = state.clone()
        want[0] = 0
        assert out.shape == (0, 2, 64) and torch.equal(layer.state.cpu(), want) and int(layer.status.item()) == 0


def test_many_tokens_that_empty_the_state():
    """Decays of the lowest value add up to thousands in a chunk; what is left between them is still exact to a bf16."""
    T, Hv = 300, 4
    row, _ = inputs((T,), 1, Hv, 64, 64, 12, True)
    g = torch.Generator().manual_seed(13)
    decay = -0.05 * torch.rand((T, Hv), generator=g)
    decay[:64, 0] = -math.inf
    decay[::2, 1] = -math.inf
    decay[torch.rand(T, generator=g) < 0.7, 2] = -200.0
    decay[:120, 3] = -104.0
    run_prompts([T], 1, Hv, 64, 64, True, [1], row=row, decay=decay)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_many_heads(dk, dv):
    """Heads enough that a piece of the work adds up the sums before it by itself: long sequences cut into several
    pieces, short ones that need no sums, continued ones, decays that empty the state, an infinity on the way."""
    lens, Hk, Hv = [900, 1, 130, 3, 0, 40, 1300, 257], 8, 16
    init = [1, 0, 1, 0, 1, 1, 0, 1]
    row, decay = inputs((sum(lens),), Hk, Hv, dk, dv, 60, True, rate=0.02)
    for t, h in ((10, 0), (899, 1), (500, 2), (1200, 3), (1201, 3), (2300, 4)):
        decay[t, h] = -math.inf
    _, layer = run_prompts(lens, Hk, Hv, dk, dv, True, init, seed=60, row=row, decay=decay)
    assert int(layer.status.item()) == 0
    run_prompts([2600], Hk, Hv, dk, dv, False, None, seed=61, rate=0.01)


def test_many_heads_again_and_beside_each_other():
    """Heads enough as above: the same bits again, in two graphs replayed beside each other, and calls in a row that
    continue each other's states; a value that is not finite reaches its own column only."""
    Hk, Hv, d, T = 8, 16, 128, 1500
    row, decay = inputs((T + 60,), Hk, Hv, d, d, 70, True, rate=0.02)
    q, k, v = views(row.cuda(), Hk, Hv, d, d)
    g = decay.cuda()
    cu = torch.tensor([0, 20, T, T + 60], dtype=torch.int32, device="cuda")
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    init = torch.tensor([1, 1, 0], dtype=torch.uint8, device="cuda")

    def calls(layer, out):
        for i in range(4):
            layer.prefill(cu, slots, init if i else None, q, k, v, g, out=out)
    layers = [runtime.DecayAttention(Hk, Hv, d, d, 3) for _ in range(4)]
    outs = [torch.zeros((T + 60, Hv, d), dtype=torch.bfloat16, device="cuda") for _ in layers]
    calls(layers[0], outs[0])
    calls(layers[1], outs[1])
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for layer, o, s in zip(layers[2:], outs[2:], streams):
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            calls(layer, o)
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for layer, o in zip(layers[1:], outs[1:]):
        assert torch.equal(o, outs[0]) and torch.equal(layer.state, layers[0].state)
    for t, value in ((21, math.nan), (700, math.inf)):
        spoiled = v.clone()
        spoiled[t, 5, 9] = value
        layer, clean = runtime.DecayAttention(Hk, Hv, d, d, 3), runtime.DecayAttention(Hk, Hv, d, d, 3)
        got = layer.prefill(cu, slots, None, q, k, spoiled, g)
        want = clean.prefill(cu, slots, None, q, k, v, g)
        assert not bool(got[t:T, 5, 9].isfinite().any()) and not bool(layer.state[1, 5, :, 9].isfinite().any())
        got[t:T, 5, 9], want[t:T, 5, 9], layer.state[1, 5, :, 9], clean.state[1, 5, :, 9] = 0, 0, 0, 0
        assert torch.equal(got, want) and torch.equal(layer.state, clean.state)
