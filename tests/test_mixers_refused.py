"""Host checks of the mixers' calls: what they refuse, before any CUDA call; the magnitude of scaled rotations."""
import ctypes
import math

import pytest
import torch

from gated_deltanet_linear_09_gb300 import build as gbuild
from gated_deltanet_linear_09_gb300 import gdn, runtime

A = 0x10000
INV = -1


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load()


def test_tokens_of_no_sequence(monkeypatch):
    """Tokens without a sequence have no output: refused, as by the library; nothing at all is nothing."""
    monkeypatch.setattr(gdn, "load", lambda: pytest.fail("the library was called"))
    layer = runtime.DecayAttention(1, 2, 64, 64, 3, device="cpu")
    cu, slots, g = torch.zeros(1, dtype=torch.int32), torch.zeros(0, dtype=torch.int32), torch.zeros(2)
    q, v = torch.zeros((5, 1, 64), dtype=torch.bfloat16), torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        layer.prefill(cu, slots, None, q, q, v, g)
    assert layer.prefill(cu, slots, None, q[:0], q[:0], v[:0], g).shape == (0, 2, 64)


@pytest.mark.parametrize("name", ["x", "gate", "residual"])
@pytest.mark.parametrize("out", ["total", "y"])
def test_block_outputs_in_place_of_strided_inputs(lib, name, out):
    """A dense output in the place of rows that lie further apart would overwrite rows that are still to be read."""
    d = dict(x=A, gate=2 * A, residual=3 * A, post=4 * A, pre=5 * A, x_ld=256, gate_ld=256, residual_ld=256, total=6 * A, y=7 * A,
             scale=1.0, weight_offset=1.0, eps=1e-6, group=256, gate_act=gdn.GDN_GATE_SILU)
    a = gdn.gdn_block_args(**{**d, out: d[name], f"{name}_ld": 264})
    assert lib.gdn_block_norm(ctypes.byref(a), 2, 256, gdn.GDN_BF16, None) == INV


def test_outputs_in_place_of_the_other_input(lib):
    """Queries' output in the place of the keys, or the other way round, or both outputs in one place."""
    r = gdn.gdn_rotary(turns=A, rot_dim=64, interleaved=0, scale=1.0)
    for q_out, k_out in ((2 * A, 4 * A), (3 * A, A), (3 * A, 3 * A)):
        assert lib.gdn_rotary_apply(ctypes.byref(r), A, 2, 128, gdn.GDN_BF16, A, 256, 128, 2, q_out, 2 * A, 256, 128, 2, k_out, None) == INV
    c = gdn.gdn_kv_cache(A, A, None, None, 4, 16, 2, 128, gdn.GDN_KV_BF16, None)
    b = gdn.gdn_kv_batch(cu_seqlens=A, kv_lens=A, block_table=A, num_seqs=1, total_tokens=1, table_ld=4, max_tokens=1)
    p = gdn.gdn_head_prep(A, A, 1.0, 1e-6, None)
    for q_out in (2 * A, 3 * A):
        assert lib.gdn_kv_append_rotated(ctypes.byref(c), ctypes.byref(b), ctypes.byref(r), ctypes.byref(p), A, 512, 128, 4, q_out, 2 * A,
                                         256, 3 * A, 256, None) == INV


@pytest.mark.parametrize("factor", [0.5, 1.0, 1.5, 8.0])
def test_magnitude_of_scaled_bands(factor):
    """0.1 ln(factor) + 1 of a stretched context; 1 where nothing is stretched."""
    plan = runtime.Rotary(64, 1e4, scaling="bands", factor=factor, trained=4096, device="cpu")
    assert plan.scale == (pytest.approx(0.1 * math.log(factor) + 1.0) if factor > 1.0 else 1.0)


def test_rotary_output_without_its_input(monkeypatch):
    """It would be returned unwritten."""
    monkeypatch.setattr(gdn, "load", lambda: pytest.fail("the library was called"))
    plan, pos, x = runtime.Rotary(64, device="cpu"), torch.zeros(3, dtype=torch.int32), torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    for args in (dict(q_out=x), dict(k_out=x), dict(q=x, k_out=x), dict(k=x, q_out=x)):
        with pytest.raises(ValueError):
            plan.apply(pos, **args)
    assert plan.apply(pos) == (None, None)
