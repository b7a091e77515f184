"""Out-of-bounds write checks of the norm, cache and attention calls: outputs, pages and the
workspace sit between canary regions, and places that no new token has keep their bytes."""
import pytest
import torch

import paged_ref as ref
from gated_deltanet_linear_09_gb300 import gdn, runtime
from gpu_util import Guarded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,n,act,kind", [(5, 131, torch.bfloat16, gdn.GDN_NORM_ACT), (3, 1000, torch.float32, gdn.GDN_NORM_ACT),
                                             (7, 4096, torch.bfloat16, gdn.GDN_NORM_E4M3_BLOCK),
                                             (9, 2047, torch.bfloat16, gdn.GDN_NORM_E4M3_ROW), (2, 20000, torch.bfloat16, gdn.GDN_NORM_E4M3_BLOCK)])
def test_norm_writes_inside(rows, n, act, kind):
    x, r, w = (torch.randn(s, device="cuda").to(act) for s in ((rows, n), (rows, n), (n,)))
    y = Guarded((rows, n), act if kind == gdn.GDN_NORM_ACT else torch.float8_e4m3fn)
    total = Guarded((rows, n), act)
    scales = None if kind == gdn.GDN_NORM_ACT else Guarded((rows, 1 if kind == gdn.GDN_NORM_E4M3_ROW else -(-n // 128)), torch.float32)
    gdn.gdn_rms_norm(x, w, y.view, r, total.view, None if scales is None else scales.view, 0.0, 1e-6, kind)
    for g in (y, total, scales):
        if g is not None:
            g.check()


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("dim,new,group", [(64, 1, 4), (128, 2, 8), (256, 1, 8), (64, 9, 8), (128, 40, 4), (256, 30, 8)])
def test_cache_and_attention_write_inside(dim, new, group, quantised):
    case = ref.Case([new, 0, 1, new + 3], [new + 333, 5, 1, new + 3], 2, dim, 16, quantised, seed=21, pad_tokens=2)
    src = case.filled_cache(runtime)
    guards = [Guarded(tuple(t.shape), t.dtype) for t in (src.k_pages, src.v_pages)]
    scales = [Guarded(tuple(t.shape), t.dtype) for t in (src.k_scales, src.v_scales)] if quantised else [None, None]
    for g, t in zip(guards + scales, (src.k_pages, src.v_pages, src.k_scales, src.v_scales)):
        if g is not None:
            g.view.view(torch.uint8).copy_(t.view(torch.uint8))
    cache = runtime.PagedKVCache.over(guards[0].view, guards[1].view, *(None if g is None else g.view for g in scales))
    b = case.device_batch(runtime)
    T = b.total_tokens
    kv = torch.randn((T, 2, dim), device="cuda").to(torch.bfloat16)
    cache.append(b, kv, kv)
    own = torch.zeros((case.num_pages, case.page), dtype=torch.bool)
    for i, (a, t) in enumerate(zip(case.new, case.lens)):
        for p in range(t - a, t):
            own[int(case.table[i, p // case.page]), p % case.page] = True
    for t, u in ((cache.k_pages, src.k_pages), (cache.v_pages, src.v_pages)):
        same = (t.view(torch.uint8) == u.view(torch.uint8)).all(-1).all(1).cpu()      # [pages][page_size]
        assert same[~own].all()
    k, v, out = Guarded((T, 2, dim), torch.bfloat16), Guarded((T, 2, dim), torch.bfloat16), Guarded((T, 2 * group, dim), torch.bfloat16)
    cache.read(b, k.view, v.view)
    ws = Guarded((gdn.gdn_paged_attention_workspace_bytes(cache.c, 2 * group),), torch.uint8)
    q = torch.randn((T, 2 * group, dim), device="cuda").to(torch.bfloat16)
    cache.attend(b, q, gate=q, out=out.view, workspace=ws.view)
    for g in [k, v, out, ws] + guards + [s for s in scales if s is not None]:
        g.check()
    assert int(cache.status.item()) == 0
