"""Tensors whose dimensions of size one have strides of their own."""
import pytest
import torch

import paged_ref as ref
from gated_deltanet_linear_09_gb300 import runtime

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quantised", [False, True])
def test_one_token_in_head_major_order(quantised):
    """[heads][1][dim] transposed: appended and attended as the dense tensor is."""
    case = ref.Case([1], [40], 2, 128, 16, quantised, seed=71)
    b = case.device_batch(runtime)
    kv = torch.randn((2, 1, 128), device="cuda").to(torch.bfloat16)
    q = torch.randn((8, 1, 128), device="cuda").to(torch.bfloat16)
    got = []
    for form in (lambda t: t.transpose(0, 1), lambda t: t.transpose(0, 1).contiguous()):
        cache = case.filled_cache(runtime)
        cache.append(b, form(kv), form(-kv))
        got.append((*cache.read(b), cache.attend(b, form(q), gate=form(q))))
        assert int(cache.status.item()) == 0
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("new", [3, 60])
def test_one_head(new):
    """One key/value head and one query head, as views with a stride of their own."""
    case = ref.Case([new], [new + 30], 1, 64, 16, False, seed=72)
    b = case.device_batch(runtime)
    x = torch.randn((new, 1, 64), device="cuda").to(torch.bfloat16)
    odd = x.as_strided((new, 1, 64), (64, 3, 1))
    got = []
    for t in (odd, x):
        cache = case.filled_cache(runtime)
        cache.append(b, t, t)
        got.append((*cache.read(b), cache.attend(b, t, gate=t)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
