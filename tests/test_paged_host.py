"""Host checks of the norm, cache and attention calls: every refusal comes before any CUDA call
(the addresses are never dereferenced), and the 64-bit forms the GPU tests use are what they say."""
import ctypes

import pytest
import torch

import paged_ref as ref
from gated_deltanet_linear_09_gb300 import build as gbuild
from gated_deltanet_linear_09_gb300 import gdn

A = 0x10000
INV, SHAPE, DIV, SMALL, ALIGN, LARGE = -1, -2, -3, -5, -7, -9


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load()


def cache(**kw):
    d = dict(k_pages=A, v_pages=A, k_scales=None, v_scales=None, num_pages=4, page_size=16, num_kv_heads=2,
             head_dim=128, type=gdn.GDN_KV_BF16, status=None)
    d.update(kw)
    return gdn.gdn_kv_cache(**d)


def batch(**kw):
    d = dict(cu_seqlens=A, kv_lens=A, block_table=A, num_seqs=1, total_tokens=1, table_ld=4, max_tokens=1)
    d.update(kw)
    return gdn.gdn_kv_batch(**d)


BAD_CACHES = [
    (dict(head_dim=96), SHAPE), (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE),
    (dict(page_size=512), SHAPE), (dict(num_kv_heads=0), INV), (dict(num_pages=0), INV), (dict(type=7), INV),
    (dict(k_pages=None), INV), (dict(k_scales=A, v_scales=A), INV), (dict(type=gdn.GDN_KV_E4M3), INV),
    (dict(type=gdn.GDN_KV_E4M3, k_scales=A), INV), (dict(v_pages=A + 8), ALIGN),
    (dict(type=gdn.GDN_KV_E4M3, k_scales=A, v_scales=A + 8), ALIGN),
]
BAD_BATCHES = [
    (dict(num_seqs=-1), INV), (dict(total_tokens=-1), INV), (dict(table_ld=-1), INV), (dict(max_tokens=-1), INV),
    (dict(num_seqs=70000), LARGE), (dict(num_seqs=0), INV), (dict(cu_seqlens=None), INV), (dict(kv_lens=None), INV),
    (dict(block_table=None), INV), (dict(kv_lens=A + 2), ALIGN),
]


def test_cache_and_batch_refusals(lib):
    def append(c, b, k_ld=256, k=A):
        return lib.gdn_kv_append(ctypes.byref(c), ctypes.byref(b), k, k_ld, A, 256, None)

    def read(c, b, k=A):
        return lib.gdn_kv_read(ctypes.byref(c), ctypes.byref(b), k, A, None)

    def attend(c, b):
        return lib.gdn_paged_attention(ctypes.byref(c), ctypes.byref(b), 8, A, 1024, 128, None, 0, 0, 0.0, A, A,
                                       1 << 40, None)
    for kw, code in BAD_CACHES:
        for call in (append, read, attend):
            assert call(cache(**kw), batch()) == code, (call.__name__, kw)
    for kw, code in BAD_BATCHES:
        for call in (append, read, attend):
            assert call(cache(), batch(**kw)) == code, (call.__name__, kw)
    assert append(cache(), batch(), k_ld=255) == INV
    assert append(cache(), batch(), k_ld=260) == ALIGN
    assert append(cache(), batch(), k=None) == INV
    assert append(cache(), batch(), k=A + 2) == ALIGN
    assert read(cache(), batch(), k=A + 2) == ALIGN
    assert append(cache(), batch(total_tokens=0), k=None) == 0
    assert read(cache(), batch(total_tokens=0), k=None) == 0
    assert lib.gdn_kv_append(None, ctypes.byref(batch()), A, 256, A, 256, None) == INV
    assert lib.gdn_kv_append(ctypes.byref(cache()), None, A, 256, A, 256, None) == INV


def test_attention_refusals(lib):
    def attend(b=None, Hq=8, q=A, q_ld=1024, q_hs=128, gate=None, g_ld=0, g_hs=0, scale=0.0, out=A, ws=A,
               nbytes=1 << 40):
        return lib.gdn_paged_attention(ctypes.byref(cache()), ctypes.byref(b or batch()), Hq, q, q_ld, q_hs, gate, g_ld,
                                       g_hs, scale, out, ws, nbytes, None)
    need = gdn.gdn_paged_attention_workspace_bytes(cache(), 8)
    assert need > 0
    assert attend(Hq=0) == INV and attend(Hq=7) == DIV
    assert attend(scale=-1.0) == INV and attend(scale=float("nan")) == INV and attend(scale=float("inf")) == INV
    assert attend(q=None) == INV and attend(out=None) == INV
    assert attend(q_ld=64) == INV and attend(q_hs=64) == INV
    assert attend(q=A + 2) == ALIGN and attend(out=A + 8) == ALIGN and attend(q_ld=1028) == ALIGN
    assert attend(gate=A) == INV
    assert attend(gate=A, g_ld=1024, g_hs=132) == ALIGN
    assert attend(gate=A + 8, g_ld=1024, g_hs=128) == ALIGN
    assert attend(ws=None) == SMALL and attend(nbytes=need - 1) == SMALL and attend(ws=A + 16) == ALIGN
    assert attend(b=batch(total_tokens=(1 << 27) + 1)) == LARGE
    assert attend(b=batch(total_tokens=0), q=None) == 0
    assert gdn.gdn_paged_attention_workspace_bytes(cache(head_dim=96), 8) == 0
    assert gdn.gdn_paged_attention_workspace_bytes(cache(), 7) == 0


def test_norm_refusals(lib):
    def norm(x=A, x_ld=64, r=None, r_ld=0, w=A, eps=1e-6, rows=2, n=64, act=gdn.GDN_BF16, kind=0, y=A, s=None,
             off=0.0):
        return lib.gdn_rms_norm(x, x_ld, r, r_ld, w, off, eps, rows, n, act, kind, None, y, s, None)
    assert norm(act=5) == INV and norm(kind=3) == INV and norm(rows=-1) == INV and norm(n=0) == INV
    assert norm(n=gdn.GDN_MAX_NORM_WIDTH + 1, x_ld=1 << 20) == LARGE
    assert norm(eps=-1.0) == INV and norm(eps=float("nan")) == INV and norm(off=float("inf")) == INV
    assert norm(x=None) == INV and norm(w=None) == INV and norm(y=None) == INV and norm(kind=1) == INV
    assert norm(x_ld=63) == INV and norm(r=A, r_ld=63) == INV
    assert norm(x=A + 8) == ALIGN and norm(kind=2, s=A + 4) == ALIGN
    assert norm(rows=0, x=None) == 0


def test_reference_quantiser():
    """The 64-bit e4m3 rounding of the tests equals torch's cast on every code and halfway point."""
    codes = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(ref.E4M3).double()
    v = torch.sort(codes[torch.isfinite(codes)]).values
    mid = (v[1:] + v[:-1]) / 2
    x = torch.cat([v, mid, mid * (1 + 2.0 ** -12), mid * (1 - 2.0 ** -12)])
    assert torch.equal(ref.e4m3_round(x), x.float().to(ref.E4M3).double())
    x = torch.tensor([[448.0], [448.1], [1.0], [0.0], [2.0 ** -130]], dtype=torch.float64)
    assert ref.scale_exponent(x).tolist() == [0.0, 1.0, -8.0, 0.0, -117.0]
