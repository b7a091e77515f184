"""Host checks of the rotary, rotated append, block norm and decayed attention calls: every refusal comes before
any CUDA call (the addresses are never dereferenced); and which tensors the Python calls take."""
import ctypes
import math

import pytest
import torch

import mixer_ref as mr
from gated_deltanet_linear_09_gb300 import build as gbuild
from gated_deltanet_linear_09_gb300 import gdn, runtime

A = 0x10000
INV, SHAPE, DIV, SMALL, ALIGN, LARGE = -1, -2, -3, -5, -7, -9
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load()


def rot(**kw):
    return gdn.gdn_rotary(**{**dict(turns=A, rot_dim=64, interleaved=0, scale=1.0), **kw})


def test_rotary_refusals(lib):
    def call(r=None, pos=A, tokens=2, dim=128, act=gdn.GDN_BF16, q=A, q_ld=512, q_hs=128, Hq=4, qo=A, k=A, k_ld=128, k_hs=128, Hk=1, ko=A):
        return lib.gdn_rotary_apply(ctypes.byref(r or rot()), pos, tokens, dim, act, q, q_ld, q_hs, Hq, qo, k, k_ld, k_hs, Hk, ko, None)
    assert call(act=3) == INV and call(tokens=-1) == INV and call(dim=0) == INV and call(Hq=-1) == INV and call(Hk=-1) == INV
    assert call(rot(scale=NAN)) == INV and call(rot(scale=INF)) == INV
    assert call(rot(rot_dim=0)) == SHAPE and call(rot(rot_dim=63)) == SHAPE and call(rot(rot_dim=130)) == SHAPE
    assert call(dim=1025) == LARGE and call(Hq=65537) == LARGE and call(Hk=65537) == LARGE
    assert call(rot(turns=None)) == INV and call(pos=None) == INV and call(q=None) == INV and call(qo=None) == INV
    assert call(k=None) == INV and call(ko=None) == INV and call(q_ld=127) == INV and call(q_hs=127) == INV and call(k_ld=127) == INV
    assert call(rot(turns=A + 4)) == ALIGN and call(pos=A + 2) == ALIGN and call(q=A + 1) == ALIGN and call(ko=A + 1) == ALIGN
    assert call(act=gdn.GDN_F32, q=A + 2) == ALIGN
    assert call(tokens=0, q=None, pos=None) == 0 and call(Hq=0, Hk=0, q=None, k=None) == 0
    assert lib.gdn_rotary_apply(None, A, 1, 64, 1, A, 64, 64, 1, A, None, 0, 0, 0, None, None) == INV


def test_append_rotated_refusals(lib):
    def call(r=None, prep=None, cache=None, batch=None, q=A, q_ld=512, q_hs=128, Hq=4, qo=A, k=A, k_ld=256, v=A, v_ld=256):
        c = gdn.gdn_kv_cache(**{**dict(k_pages=A, v_pages=A, k_scales=None, v_scales=None, num_pages=4, page_size=16, num_kv_heads=2,
                                       head_dim=128, type=gdn.GDN_KV_BF16, status=None), **(cache or {})})
        b = gdn.gdn_kv_batch(**{**dict(cu_seqlens=A, kv_lens=A, block_table=A, num_seqs=1, total_tokens=1, table_ld=4, max_tokens=1),
                                **(batch or {})})
        p = gdn.gdn_head_prep(**{**dict(q_norm=A, k_norm=A, weight_offset=1.0, eps=1e-6, positions=None), **(prep or {})})
        return lib.gdn_kv_append_rotated(ctypes.byref(c), ctypes.byref(b), ctypes.byref(r or rot()), ctypes.byref(p), q, q_ld, q_hs, Hq, qo,
                                         k, k_ld, v, v_ld, None)
    assert call(cache=dict(head_dim=96)) == SHAPE and call(cache=dict(k_pages=None)) == INV and call(batch=dict(num_seqs=0)) == INV
    assert call(batch=dict(kv_lens=A + 2)) == ALIGN
    for bad in (dict(weight_offset=INF), dict(eps=-1.0), dict(eps=NAN)):
        assert call(prep=bad) == INV
    assert call(rot(scale=INF)) == INV and call(Hq=-1) == INV and call(Hq=(1 << 20) + 1, q_ld=1 << 40) == LARGE
    assert call(rot(rot_dim=8)) == SHAPE and call(rot(rot_dim=72)) == SHAPE and call(rot(rot_dim=144)) == SHAPE
    assert call(k_ld=255) == INV and call(v_ld=255) == INV and call(q_ld=64) == INV and call(q_hs=64) == INV
    assert call(k=None) == INV and call(v=None) == INV and call(q=None) == INV and call(qo=None) == INV and call(rot(turns=None)) == INV
    assert call(rot(turns=A + 4)) == ALIGN and call(prep=dict(positions=A + 2)) == ALIGN and call(prep=dict(q_norm=A + 8)) == ALIGN
    assert call(k=A + 8) == ALIGN and call(v_ld=260) == ALIGN and call(q_hs=132) == ALIGN and call(qo=A + 4) == ALIGN
    assert call(batch=dict(total_tokens=0), k=None, q=None) == 0
    assert lib.gdn_kv_append_rotated(None, None, None, None, A, 1, 1, 1, A, A, 1, A, 1, None) == INV


def test_block_refusals(lib):
    def call(rows=2, n=256, act=gdn.GDN_BF16, **kw):
        d = dict(x=A, gate=A, residual=A, post=A, pre=A, channel_scale=A, x_ld=256, gate_ld=256, residual_ld=256, total=A, y=A,
                 scale=1.0, weight_offset=1.0, eps=1e-6, group=64, gate_act=gdn.GDN_GATE_SILU)
        return lib.gdn_block_norm(ctypes.byref(gdn.gdn_block_args(**{**d, **kw})), rows, n, act, None)
    assert call(rows=-1) == INV and call(n=0) == INV and call(act=2) == INV and call(gate_act=3) == INV
    assert call(eps=-1.0) == INV and call(eps=NAN) == INV and call(scale=INF) == INV and call(weight_offset=NAN) == INV
    assert call(n=gdn.GDN_MAX_NORM_WIDTH + 1) == LARGE
    assert call(group=48) == SHAPE and call(group=512) == SHAPE and call(group=0) == SHAPE and call(n=255, group=64) == SHAPE
    assert call(x=None) == INV and call(gate=None) == INV and call(gate_act=0) == INV and call(pre=None) == INV and call(y=None) == INV
    assert call(pre=None, y=None, total=None) == INV
    assert call(x_ld=255) == INV and call(gate_ld=255) == INV and call(residual_ld=255) == INV
    for name in ("x", "gate", "residual", "post", "pre", "channel_scale", "total", "y"):
        assert call(**{name: A + 8}) == ALIGN, name
    assert call(x_ld=260) == ALIGN and call(gate_ld=257) == ALIGN
    assert call(rows=0, x=None) == 0 and lib.gdn_block_norm(None, 1, 8, 1, None) == INV


def test_decay_refusals(lib):
    def parts(layer, tokens):
        l = gdn.gdn_decay_layer(**{**dict(state=A, num_slots=4, num_k_heads=2, num_v_heads=4, head_k_dim=128, head_v_dim=64, scale=0.0,
                                          status=None), **(layer or {})})
        t = gdn.gdn_decay_tokens(**{**dict(q=A, k=A, v=A, q_ld=256, k_ld=256, v_ld=256, log_decay=A, decay_ld=4, out=A), **(tokens or {})})
        return ctypes.byref(l), ctypes.byref(t)

    def step(layer=None, tokens=None, slots=A, B=2, T=1):
        return lib.gdn_decay_step(*parts(layer, tokens), slots, B, T, None)

    def prefill(layer=None, tokens=None, slots=A, cu=A, n=2, total=10, ws=A, nbytes=1 << 40):
        return lib.gdn_decay_prefill(*parts(layer, tokens), cu, slots, None, n, total, ws, nbytes, None)
    for call in (step, prefill):
        for bad, code in ((dict(num_k_heads=0), INV), (dict(num_v_heads=0), INV), (dict(num_v_heads=5), DIV), (dict(head_k_dim=96), SHAPE),
                          (dict(head_v_dim=256), SHAPE), (dict(scale=-1.0), INV), (dict(scale=NAN), INV), (dict(state=None), INV),
                          (dict(num_slots=0), INV), (dict(state=A + 8), ALIGN), (dict(num_k_heads=1, num_v_heads=65536), LARGE)):
            assert call(layer=bad) == code, (call.__name__, bad)
        for bad, code in ((dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(out=None), INV), (dict(log_decay=None), INV),
                          (dict(q_ld=255), INV), (dict(k_ld=128), INV), (dict(v_ld=248), INV), (dict(decay_ld=3), INV),
                          (dict(decay_ld=-4), INV), (dict(q=A + 8), ALIGN), (dict(out=A + 2), ALIGN), (dict(log_decay=A + 2), ALIGN),
                          (dict(v_ld=260), ALIGN)):
            assert call(tokens=bad) == code, (call.__name__, bad)
        assert call(slots=None) == INV and call(slots=A + 2) == ALIGN
    assert step(T=0) == INV and step(T=gdn.GDN_MAX_DECODE_TOKENS + 1) == INV and step(B=-1) == INV and step(B=65536) == LARGE
    assert step(B=0, slots=None, tokens=dict(q=None)) == 0
    l, _ = parts(None, None)
    need = lib.gdn_decay_prefill_workspace_bytes(l, 2, 10)
    assert need > 0 and lib.gdn_decay_prefill_workspace_bytes(l, -1, 10) == 0
    assert lib.gdn_decay_prefill_workspace_bytes(parts(dict(head_k_dim=32), None)[0], 2, 10) == 0
    assert prefill(n=-1) == INV and prefill(total=-1) == INV and prefill(n=65536) == LARGE and prefill(n=0) == INV
    assert prefill(cu=None) == INV and prefill(cu=A + 2) == ALIGN
    assert prefill(ws=None) == SMALL and prefill(nbytes=need - 1) == SMALL and prefill(ws=A + 16) == ALIGN
    assert prefill(n=0, total=0, tokens=dict(q=None)) == 0
    assert lib.gdn_decay_step(None, None, A, 1, 1, None) == INV


def test_outputs_are_not_the_inputs(lib):
    """Outputs in the place of inputs, where the call cannot have them there."""
    r = rot()
    for heads, ld, head_ld, tokens in ((2, 256, 128, 2), (2, 257, 128, 2), (2, 258, 129, 2), (2, 258, 129, 1)):
        want = 0 if (ld, head_ld) == (256, 128) else INV
        if want:            # (the first would launch)
            assert lib.gdn_rotary_apply(ctypes.byref(r), A, tokens, 128, gdn.GDN_BF16, A, ld, head_ld, heads, A, None, 0, 0, 0, None, None) == want
            assert lib.gdn_rotary_apply(ctypes.byref(r), A, tokens, 128, gdn.GDN_BF16, None, 0, 0, 0, None, A, ld, head_ld, heads, A, None) == want
    c = gdn.gdn_kv_cache(A, A, None, None, 4, 16, 2, 128, gdn.GDN_KV_BF16, None)
    b = gdn.gdn_kv_batch(cu_seqlens=A, kv_lens=A, block_table=A, num_seqs=1, total_tokens=1, table_ld=4, max_tokens=1)
    p = gdn.gdn_head_prep(A, A, 1.0, 1e-6, None)
    assert lib.gdn_kv_append_rotated(ctypes.byref(c), ctypes.byref(b), ctypes.byref(r), ctypes.byref(p), A, 512, 128, 4, A, A, 256, A, 256, None) == INV
    a = gdn.gdn_block_args(x=A, pre=A, total=2 * A, y=2 * A, x_ld=256, scale=1.0, weight_offset=0.0, eps=1e-6, group=256, gate_act=0)
    assert lib.gdn_block_norm(ctypes.byref(a), 2, 256, gdn.GDN_BF16, None) == INV
    for name in ("q", "k", "v"):
        l = gdn.gdn_decay_layer(A, 4, 2, 4, 128, 64, 0.0, None)
        t = gdn.gdn_decay_tokens(**{**dict(q=A, k=A, v=A, q_ld=256, k_ld=256, v_ld=256, log_decay=A, decay_ld=4, out=2 * A), name: 2 * A})
        assert lib.gdn_decay_step(ctypes.byref(l), ctypes.byref(t), A, 2, 1, None) == INV
        assert lib.gdn_decay_prefill(ctypes.byref(l), ctypes.byref(t), A, A, None, 2, 10, A, 1 << 40, None) == INV


def test_structs_match_the_header():
    """Sizes as the C compiler lays them out on a 64-bit machine."""
    assert ctypes.sizeof(gdn.gdn_rotary) == 24 and ctypes.sizeof(gdn.gdn_head_prep) == 32
    assert ctypes.sizeof(gdn.gdn_block_args) == 8 * 6 + 24 + 16 + 12 + 8 + 4
    assert ctypes.sizeof(gdn.gdn_decay_layer) == 40 and ctypes.sizeof(gdn.gdn_decay_tokens) == 72


def test_frequencies():
    """Unscaled, divided, stretched by the base and by bands, against their definitions; turns modulo one."""
    r, base = 64, 1e4
    f = [base ** (-2 * i / r) for i in range(r // 2)]
    plan = runtime.Rotary(r, base, device="cpu")
    assert plan.frequencies == pytest.approx(f, rel=1e-14) and plan.scale == 1.0
    for t, x in zip(plan.turns.tolist(), f):
        assert t % 2 ** 64 / 2 ** 64 == pytest.approx(x / (2 * math.pi) % 1, abs=2 ** -52)
    assert runtime.Rotary(r, base, scaling="linear", factor=4.0, device="cpu").frequencies == pytest.approx([x / 4 for x in f])
    stretched = runtime.Rotary(r, base, scaling="base", factor=8.0, device="cpu").frequencies
    assert stretched[0] == 1.0 and stretched[-1] == pytest.approx(f[-1] / 8.0)
    bands = runtime.Rotary(r, base, scaling="bands", factor=8.0, trained=4096, device="cpu")
    for x, y in zip(bands.frequencies, f):
        turns = 4096 * y / (2 * math.pi)
        if turns > 40:
            assert x == pytest.approx(y)
        elif turns < 0.8:
            assert x == pytest.approx(y / 8)
        else:
            assert y / 8 * (1 - 1e-9) <= x <= y * (1 + 1e-9)
    assert bands.scale == pytest.approx(0.1 * math.log(8.0) + 1.0)
    assert runtime.Rotary.of([0.5, 7.0], scale=2.0, device="cpu").turns.tolist()[1] % 2 ** 64 / 2 ** 64 == pytest.approx(7 / (2 * math.pi) - 1)
    for bad in (lambda: runtime.Rotary(7), lambda: runtime.Rotary(0), lambda: runtime.Rotary(8, base=1.0), lambda: runtime.Rotary(8, factor=0.0),
                lambda: runtime.Rotary(8, scaling="other", device="cpu"), lambda: runtime.Rotary.of([], device="cpu"),
                lambda: runtime.Rotary.of([INF], device="cpu")):
        with pytest.raises(ValueError):
            bad()


def test_python_calls_refuse(monkeypatch):
    """Wrong shapes, types, strides and devices are refused before the library is reached; host memory too."""
    monkeypatch.setattr(gdn, "load", lambda: pytest.fail("the library was called"))
    bf = dict(dtype=torch.bfloat16)
    x, w = torch.zeros((4, 64), **bf), torch.zeros(64, **bf)
    meta = torch.zeros((4, 64), device="meta", **bf)
    plan = runtime.Rotary(32, device="cpu")
    pos = torch.zeros(4, dtype=torch.int32)
    h = torch.zeros((4, 2, 64), **bf)
    cache = runtime.PagedKVCache(4, 16, 2, 64, device="cpu")
    i32 = dict(dtype=torch.int32)
    batch = runtime.KVBatch(torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros((2, 2), **i32), 4, 2)
    layer = runtime.DecayAttention(1, 2, 64, 64, 3, device="cpu")
    q, v, g = torch.zeros((4, 1, 64), **bf), torch.zeros((4, 2, 64), **bf), torch.zeros(2)
    slots, cu = torch.zeros(4, **i32), torch.zeros(5, **i32)
    refused = [
        lambda: plan.apply(pos.long(), h), lambda: plan.apply(pos[:3], h), lambda: plan.apply(pos, h[..., :16]), lambda: plan.apply(pos, h[..., ::2]),
        lambda: plan.apply(pos, h.to("meta")), lambda: plan.apply(pos.to("meta"), h), lambda: plan.apply(pos, h, h.float()),
        lambda: plan.apply(pos, h, torch.zeros((4, 1, 32), **bf)), lambda: plan.apply(pos, h, q_out=h[:, :1]), lambda: plan.apply(pos, h),
        lambda: runtime.block_norm(x[0]), lambda: runtime.block_norm(x, gate=x[:2]), lambda: runtime.block_norm(x, residual=x.float()),
        lambda: runtime.block_norm(x, pre=w[:32]), lambda: runtime.block_norm(x, gate=x, gate_act="tanh"), lambda: runtime.block_norm(x, gate=meta),
        lambda: runtime.block_norm(x, post=w.to("meta")), lambda: runtime.block_norm(x, y=x), lambda: runtime.block_norm(x, total=x.t().contiguous().t()),
        lambda: runtime.block_norm(x, channel_scale=w.float()), lambda: runtime.block_norm(x, gate=x, gate_act="none"), lambda: runtime.block_norm(x),
        lambda: cache.append_rotated(batch, plan, h, h[:, :1], h), lambda: cache.append_rotated(batch, plan, h.float(), h, h),
        lambda: cache.append_rotated(batch, plan, h, h, h, q_norm=w.float()), lambda: cache.append_rotated(batch, plan, h, h, h, k_norm=w[:32]),
        lambda: cache.append_rotated(batch, plan, h, h, h, positions=pos.long()), lambda: cache.append_rotated(batch, plan, h, h, h, positions=pos[:2]),
        lambda: cache.append_rotated(batch, plan, None, h, h, q_out=h), lambda: cache.append_rotated(batch, plan, h, h, h, q_out=h.float()),
        lambda: cache.append_rotated(batch, runtime.Rotary(72, device="cpu"), h, h, h), lambda: cache.append_rotated(batch, runtime.Rotary(24, device="cpu"), h, h, h),
        lambda: cache.append_rotated(batch, runtime.Rotary(32, device="meta"), h, h, h), lambda: cache.append_rotated(batch, plan, h, h, h),
        lambda: runtime.DecayAttention.over(torch.zeros(2, 3, 64, 64), 2), lambda: runtime.DecayAttention.over(torch.zeros(2, 2, 64, 64).half(), 1),
        lambda: layer.step(slots.long(), q, q, v, g), lambda: layer.step(slots[:3], q, q, v, g), lambda: layer.step(slots, q, q.float(), v, g),
        lambda: layer.step(slots, q, v, v, g), lambda: layer.step(slots, q, q, v, g.double()), lambda: layer.step(slots, q, q, v, torch.zeros(3, 2)),
        lambda: layer.step(slots, q, q, v, g, out=v.float()), lambda: layer.step(slots, q, q, v.to("meta"), g), lambda: layer.step(slots, q, q, v, g),
        lambda: layer.step(slots[:2], q.view(2, 2, 1, 64), q.view(2, 2, 1, 64), torch.zeros((2, 3, 2, 64), **bf)[:, :2], g),
        lambda: layer.step(slots, q, q, torch.zeros((4, 2, 128), **bf)[..., :64], g),
        lambda: layer.prefill(cu.long(), slots, None, q, q, v, g), lambda: layer.prefill(cu[:4], slots, None, q, q, v, g),
        lambda: layer.prefill(cu, slots, slots, q, q, v, g), lambda: layer.prefill(cu, slots, None, q, q, v[None], g),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError):
            call()
        assert i >= 0


def test_plain_forms():
    """The recurrence's 64-bit form against the quadratic one, and the block's against torch's pieces."""
    g = torch.Generator().manual_seed(0)
    T, H, dk, dv = 20, 2, 4, 3
    q, k = (torch.randn((T, 1, dk), generator=g, dtype=torch.float64) for _ in range(2))
    v, decay = torch.randn((T, H, dv), generator=g, dtype=torch.float64), -torch.rand((T, H), generator=g, dtype=torch.float64)
    o, S, _, _ = mr.decay(torch.zeros(H, dk, dv, dtype=torch.float64), q, k, v, decay)
    c = torch.cumsum(decay, 0)
    for h in range(H):
        w = torch.tril(torch.exp(c[:, None, h] - c[None, :, h])) * (q[:, 0] @ k[:, 0].T)
        assert torch.allclose(o[:, h], w @ v[:, h] / 2.0, atol=1e-12)
        assert torch.allclose(S[h], (k[:, 0] * torch.exp(c[-1, h] - c[:, h])[:, None]).T @ v[:, h], atol=1e-12)
    x = torch.randn((3, 8), generator=g, dtype=torch.float64)
    h, y = mr.block(x, post=torch.zeros(4, dtype=torch.float64), pre=torch.zeros(8, dtype=torch.float64), eps=0.0, offset=1.0)
    assert torch.allclose(h.view(3, 2, 4).pow(2).mean(-1), torch.ones(3, 2, dtype=torch.float64)) and torch.allclose(y, h)
    turned = mr.rotated(x.view(3, 1, 8), [0, 1, 2], [math.pi / 2, math.pi], 1.0, True)
    assert torch.allclose(turned[1, 0, :4], torch.stack([-x[1, 1], x[1, 0], -x[1, 2], -x[1, 3]]))
