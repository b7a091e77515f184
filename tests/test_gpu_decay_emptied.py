"""What is not finite before a token that empties the state: that token's decay of zero ends its influence, wherever a
chunk or a piece of the work ends.  Against the recurrence in 64 bits, with the bounds of test_gpu_decay.py."""
import math

import pytest
import torch

import mixer_ref as mr
from gated_deltanet_linear_09_gb300 import runtime
from test_gpu_decay import inputs, out_bound, pool, views

pytestmark = pytest.mark.gpu


def check_prompts(lens, Hk, Hv, dk, dv, init, row, decay, state, slots):
    """(outputs, layer): the call, checked against the recurrence; a log decay below -105 counts as -inf, whose exp is
    not 0 in 64 bits otherwise."""
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    layer = runtime.DecayAttention.over(state.cuda(), Hk)
    flags = torch.tensor(init, dtype=torch.uint8, device="cuda")
    got = layer.prefill(torch.tensor(cu, dtype=torch.int32, device="cuda"), slots.cuda(), flags, *views(row.cuda(), Hk, Hv, dk, dv),
                        decay.cuda())
    q, k, v = (x.double() for x in views(row, Hk, Hv, dk, dv))
    g = decay.double().masked_fill(decay < -105, -math.inf)
    touched = slots.tolist()
    for i, s in enumerate(touched):
        part = slice(cu[i], cu[i + 1])
        S0 = state[s].double() if init[i] else torch.zeros(Hv, dk, dv, dtype=torch.float64)
        o, S, size, M = mr.decay(S0, q[part], k[part], v[part], g[part])
        mr.close(got[part], o, out_bound(o, size, 2.0 ** -8 + 2.0 ** -12), f"sequence {i}")
        mr.close(layer.state[s], S, 2.0 ** -14 * M, f"state of sequence {i}")
    for s in set(range(state.shape[0])) - set(touched):
        assert torch.equal(layer.state[s].cpu(), state[s])
    return got, layer


@pytest.mark.parametrize("T", [100, 128, 500])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_keys_before_an_emptying_token(T, value):
    """In one chunk, whose scores hold what is not finite; heads that are not emptied, or before it, keep it."""
    Hk, Hv, d = 1, 3, 128
    row, decay = inputs((T,), Hk, Hv, d, d, T, True, rate=0.02)
    row[10, Hk * d + 7] = value
    row[90, Hk * d + 3] = value
    decay[14, 0] = -math.inf
    decay[91, 0] = -math.inf
    decay[95, 1] = -500.0
    slots = torch.randperm(2, generator=torch.Generator().manual_seed(T))[:1].to(torch.int32)
    got, layer = check_prompts([T], Hk, Hv, d, d, [1], row, decay, pool(2, Hv, d, d, T), slots)
    assert bool(got[14:90, 0].isfinite().all()) and bool(got[91:, 0].isfinite().all()) and bool(got[95:, 1].isfinite().all())
    assert not bool(got[10:, 2].isfinite().any()) and not bool(got[10:95, 1].isfinite().any())


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("Hk,Hv", [(1, 2), (8, 16)])
def test_long_prompts_with_emptying_tokens(Hk, Hv, dk, dv):
    """In a sequence that is cut into pieces, with heads few (chained) and many (summed by the pieces): values, keys and
    a first state that are not finite, emptied in the same piece, in a later one, or not at all."""
    lens = [1500, 60, 900]
    row, decay = inputs((sum(lens),), Hk, Hv, dk, dv, 5, True, rate=0.01)
    state = pool(4, Hv, dk, dv, 5)
    slots = torch.tensor([2, 0, 3], dtype=torch.int32)
    v0 = 2 * Hk * dk
    # head 0: a value, and a first state in its column, emptied soon after
    row[5, v0 + 9], state[2, 0, 11, 9], state[2, 0, 2, 8] = math.inf, math.inf, math.nan
    decay[40, 0] = -math.inf
    # head 1: a value that is emptied pieces later, another that stays in the state
    row[300, v0 + dv + 1] = math.nan
    decay[1000, 1] = -math.inf
    row[1200, v0 + dv + 4] = -math.inf
    # a key of the last sequence, emptied in head 0 and, a chunk later, in head 1
    row[1560 + 70, Hk * dk + 3] = math.nan
    decay[1560 + 75, 0] = -math.inf
    decay[1560 + 200, 1] = -200.0
    got, layer = check_prompts(lens, Hk, Hv, dk, dv, [1, 1, 1], row, decay, state, slots)
    assert int(layer.status.item()) == 0
    assert bool(got[40:1500, 0].isfinite().all()) and bool(layer.state[2, 0].isfinite().all())
    assert bool(got[1000:1200, 1].isfinite().all()) and not bool(layer.state[2, 1, :, 4].isfinite().any())
    assert bool(got[1635:, 0].isfinite().all()) and bool(layer.state[3, :2].isfinite().all())
