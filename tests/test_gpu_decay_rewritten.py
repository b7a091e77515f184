"""Prompts in a row whose lengths, slots, flags, decays and tokens stand in buffers that a kernel rewrites right before each
call: every call reads what was written last."""
import pytest
import torch

from gated_deltanet_linear_09_gb300 import runtime
from test_gpu_decay import inputs, pool, views

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hk,Hv", [(1, 2), (8, 16)])
def test_inputs_rewritten_before_each_call(Hk, Hv):
    d, total, n = 64, 1400, 5
    plans = []
    for i, lens in enumerate(([700, 1, 129, 400, 170], [20, 900, 300, 0, 180], [1, 1, 1, 1, 1396])):
        cu = torch.tensor([sum(lens[:j]) for j in range(n + 1)], dtype=torch.int32).cuda()
        row, decay = inputs((total,), Hk, Hv, d, d, 80 + i, True, rate=0.05)
        slots = torch.randperm(n + 1, generator=torch.Generator().manual_seed(i))[:n].to(torch.int32).cuda()
        plans.append((cu, slots, torch.tensor([(i + j) % 2 for j in range(n)], dtype=torch.uint8).cuda(), row.cuda(), decay.cuda()))
    state = pool(n + 1, Hv, d, d, 9).cuda()
    own = [torch.empty_like(t) for t in plans[0]]
    want = []
    for plan in plans:                                   # each by itself
        layer = runtime.DecayAttention.over(state.clone(), Hk)
        torch.cuda.synchronize()
        out = layer.prefill(*plan[:3], *views(plan[3], Hk, Hv, d, d), plan[4])
        torch.cuda.synchronize()
        want.append((out, layer.state))
    layer, outs = runtime.DecayAttention.over(state.clone(), Hk), [torch.empty_like(want[0][0]) for _ in range(30)]
    states = [torch.empty_like(state) for _ in outs]
    torch.cuda.synchronize()
    for i, (out, after) in enumerate(zip(outs, states)):
        for mine, new in zip(own, plans[i % 3]):
            mine.copy_(new)
        layer.state.copy_(state)
        layer.prefill(*own[:3], *views(own[3], Hk, Hv, d, d), own[4], out=out)
        after.copy_(layer.state)
    torch.cuda.synchronize()
    for i, (out, after) in enumerate(zip(outs, states)):
        assert torch.equal(out, want[i % 3][0]) and torch.equal(after, want[i % 3][1]), i
    assert int(layer.status.item()) == 0
