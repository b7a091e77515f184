"""Inconsistent batches: every output row is written, and the status says so."""
import math

import pytest
import torch

import paged_ref as ref
from gated_deltanet_linear_09_gb300 import gdn, runtime

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_linear_09_gb300 import build
    build.build()
    gdn.load()


@pytest.mark.parametrize("dim,quantised,group", [(64, True, 2), (128, False, 4), (256, False, 4), (128, True, 8)])
def test_inconsistent_token_ranges_give_zeros(dim, quantised, group):
    """Rows of a sequence that ends past the packed tokens, and rows before the first sequence, see nothing;
    the other sequences are attended as ever."""
    new, lens, tokens = [3, 40], [50, 60], 43
    case = ref.Case(new, lens, 1, dim, 16, quantised, seed=51)
    g = torch.Generator().manual_seed(52)
    q = torch.randn((tokens, group, dim), generator=g).to(torch.bfloat16)
    cache = case.filled_cache(runtime)
    b = case.device_batch(runtime)
    want, spread = ref.attention(case, q)
    bound = ref.attention_bound(want, spread)
    for cu, zero, good in (([0, 3, 50], range(3, 43), range(0, 3)), ([2, 3, 43], range(0, 2), range(3, 43)),
                           ([0, 3, 2 ** 31 - 1], range(3, 43), range(0, 3)), ([-4, 3, 43], range(0, 3), range(3, 43)),
                           ([0, 50, 43], range(0, 43), ())):
        for most in (1, 3, 40):        # the host's bound decides which kernel runs
            b = runtime.KVBatch(torch.tensor(cu, dtype=torch.int32, device="cuda"), b.tensors[1], b.tensors[2], tokens, most)
            out = torch.full((tokens, group, dim), math.nan, dtype=torch.bfloat16, device="cuda")
            cache.attend(b, q.cuda(), out=out)
            got = out.cpu().double()
            assert int(cache.status.item()) == gdn.GDN_STATUS_BAD_SEQLENS, cu
            cache.status.zero_()
            assert (got[list(zero)] == 0).all(), cu
            assert (cache.read(b)[0][list(zero)] == 0).all() and int(cache.status.item()) == gdn.GDN_STATUS_BAD_SEQLENS, cu
            cache.status.zero_()
            good = list(good)
            assert ((got[good] - want[good]).abs() <= bound[good]).all(), cu


@pytest.mark.parametrize("new", [1, 30])
@pytest.mark.parametrize("quantised", [False, True])
def test_tables_that_are_views(new, quantised):
    """Columns cut out of a wider table: a length past them is reported, and no entry beside them is read;
    and one row shared by all sequences."""
    case = ref.Case([new, new], [60, 60], 1, 64, 16, quantised, seed=53, table_extra=0)
    g = torch.Generator().manual_seed(54)
    q = torch.randn((2 * new, 4, 64), generator=g).to(torch.bfloat16).cuda()
    cache = case.filled_cache(runtime)
    b = case.device_batch(runtime)
    want = cache.attend(b, q)
    wide = torch.full((2, 9), 10 ** 9, dtype=torch.int32, device="cuda")
    wide[:, 3:7] = b.tensors[2]
    view = runtime.KVBatch(b.tensors[0], b.tensors[1], wide[:, 3:7], 2 * new, new)
    assert torch.equal(cache.attend(view, q), want) and int(cache.status.item()) == 0
    short = runtime.KVBatch(b.tensors[0], b.tensors[1], wide[:, 3:6], 2 * new, new)
    assert (cache.attend(short, q) == 0).all() and int(cache.status.item()) == gdn.GDN_STATUS_BAD_SEQLENS
    cache.status.zero_()
    kv = torch.ones((2 * new, 1, 64), dtype=torch.bfloat16, device="cuda")
    pages = cache.k_pages.clone()
    cache.append(short, kv, kv)
    assert torch.equal(pages.view(torch.uint8), cache.k_pages.view(torch.uint8))
    assert (cache.read(short)[0] == 0).all() and int(cache.status.item()) == gdn.GDN_STATUS_BAD_SEQLENS
    cache.status.zero_()
    one = runtime.KVBatch(b.tensors[0], b.tensors[1], b.tensors[2][:1].expand(2, -1), 2 * new, new)
    same = runtime.KVBatch(b.tensors[0], b.tensors[1], b.tensors[2][:1].repeat(2, 1), 2 * new, new)
    assert torch.equal(cache.attend(one, q), cache.attend(same, q)) and int(cache.status.item()) == 0
