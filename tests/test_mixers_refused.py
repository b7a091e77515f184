"""Host checks of the mixers' calls: what they refuse, before any CUDA call."""
import pytest
import torch

from gated_deltanet_linear_09_gb300 import gdn, runtime


def test_tokens_of_no_sequence(monkeypatch):
    """Tokens without a sequence have no output: refused, as by the library; nothing at all is nothing."""
    monkeypatch.setattr(gdn, "load", lambda: pytest.fail("the library was called"))
    layer = runtime.DecayAttention(1, 2, 64, 64, 3, device="cpu")
    cu, slots, g = torch.zeros(1, dtype=torch.int32), torch.zeros(0, dtype=torch.int32), torch.zeros(2)
    q, v = torch.zeros((5, 1, 64), dtype=torch.bfloat16), torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        layer.prefill(cu, slots, None, q, q, v, g)
    assert layer.prefill(cu, slots, None, q[:0], q[:0], v[:0], g).shape == (0, 2, 64)
