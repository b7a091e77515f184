"""The paged cache and attention over it against plain 64-bit forms: every head dim, cache type and
page size; ragged batches with empty sequences, sequences without places, padding rows; hidden and
out-of-range garbage; strides; strings of splits; captured graphs and other streams."""
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


def _q(case, Hq, seed=5, gate=False):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((case.tokens, Hq, case.dim), generator=g) * 1.5).to(torch.bfloat16)
    z = torch.randn((case.tokens, Hq, case.dim), generator=g).to(torch.bfloat16) if gate else None
    return q, z


def _check(case, Hq, gate=False, cache=None, scale=0.0):
    q, z = _q(case, Hq, gate=gate)
    cache = case.filled_cache(runtime) if cache is None else cache
    got = cache.attend(case.device_batch(runtime), q.cuda(), None if z is None else z.cuda(), scale).cpu().double()
    want, spread = ref.attention(case, q, z, None if scale == 0.0 else scale)
    bound = ref.attention_bound(want, spread)
    assert torch.isfinite(got).all()
    err = (got - want).abs()
    worst = (err - bound).max().item() if err.numel() else -1.0
    assert worst <= 0, f"off by {err.max().item():.3e}, {worst:.3e} beyond the bound"
    assert int(cache.status.item()) == 0
    return got


SHAPES = [  # dim, quantised, page, heads, group
    (64, False, 16, 2, 4), (64, True, 32, 2, 4), (128, False, 16, 2, 1), (128, True, 16, 3, 6),
    (128, False, 64, 1, 16), (256, False, 32, 2, 8), (256, True, 16, 1, 8), (256, True, 256, 2, 3),
    (128, True, 128, 2, 8), (64, True, 16, 1, 1),
]


@pytest.mark.parametrize("dim,quantised,page,heads,group", SHAPES)
def test_append_and_read(dim, quantised, page, heads, group):
    case = ref.Case([1, 0, 37, 5, 130], [1, 9, 37, 300, 131], heads, dim, page, quantised, seed=1, pad_tokens=3)
    cache = case.filled_cache(runtime)
    k, v = cache.read(case.device_batch(runtime))
    K, V = case.held()
    for got, want in ((k, K), (v, V)):
        got = got.cpu().double()
        for i, a in enumerate(case.new):
            assert torch.equal(got[case.cu[i]:case.cu[i + 1]], want[i][case.lens[i] - a:])
        assert (got[case.cu[-1]:] == 0).all()
    assert int(cache.status.item()) == 0


@pytest.mark.parametrize("dim,quantised,page,heads,group", SHAPES)
def test_decode(dim, quantised, page, heads, group):
    case = ref.Case([1] * 7, [1, 15, 16, 17, 64, 65, 777], heads, dim, page, quantised, seed=2)
    _check(case, heads * group, gate=group > 3)


@pytest.mark.parametrize("dim,quantised,page,heads,group", SHAPES)
def test_chunks(dim, quantised, page, heads, group):
    case = ref.Case([3, 0, 1, 33, 8, 150], [3, 40, 1, 33, 200, 1000], heads, dim, page, quantised, seed=3, pad_tokens=2)
    got = _check(case, heads * group, gate=group > 3)
    assert (got[case.cu[-1]:] == 0).all()


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_sequence_is_split(dim, quantised):
    """One sequence and head: the work can only be split along the cache."""
    case = ref.Case([1], [9001], 1, dim, 64, quantised, seed=4)
    _check(case, 4)


@pytest.mark.parametrize("new", [3, 5, 15, 16, 17])
@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
def test_rows_around_a_block(dim, quantised, new):
    """Between 17 and 136 rows under a key/value head, from one tile of keys to many."""
    case = ref.Case([new, 1, new - 1, 2], [new + 2500, 90, new - 1, 129], 2, dim, 32, quantised, seed=15, pad_tokens=1)
    got = _check(case, 16, gate=new == 16)
    assert (got[case.cu[-1]:] == 0).all()


def test_rows_that_see_nothing_are_zero():
    """More new tokens than cached positions: the first ones have no place and see no key."""
    for quantised in (False, True):
        case = ref.Case([5, 2, 4], [3, 0, 4], 2, 128, 16, quantised, seed=6)
        got = _check(case, 8, gate=True)
        assert (got[0:2] == 0).all() and (got[5:7] == 0).all()


def test_many_short_sequences():
    case = ref.Case([1] * 700, [1 + i % 40 for i in range(700)], 1, 64, 16, False, seed=7)
    _check(case, 2)


def test_hidden_values_have_no_influence():
    """NaN and infinities at positions that later tokens see and earlier ones do not."""
    for dim, quantised, new in ((128, False, 6), (256, False, 3), (128, True, 6), (64, False, 90), (256, True, 200)):
        case = ref.Case([new], [new + 20], 1, dim, 16, quantised, seed=8)
        q, _ = _q(case, 2)
        want, spread = ref.attention(case, q)
        bound = ref.attention_bound(want, spread)[:new - 2]
        bad = new + 20 - 2                     # seen by the last two tokens only
        case.v[0][bad, 0, 3] = math.nan
        case.k[0][bad, 0, 5] = math.inf
        got = case.filled_cache(runtime).attend(case.device_batch(runtime), q.cuda())
        assert ((got[:new - 2].cpu().double() - want[:new - 2]).abs() <= bound).all()
        assert torch.isnan(got[new - 2:]).any()
        # an infinite value alone reaches exactly its column
        case.k[0][bad, 0, 5] = 1.0
        case.v[0][bad, 0, 3] = math.inf
        got = case.filled_cache(runtime).attend(case.device_batch(runtime), q.cuda())
        assert ((got[:new - 2].cpu().double() - want[:new - 2]).abs() <= bound).all()
        assert not torch.isfinite(got[new - 2:, :, 3]).any()


def test_extreme_scores():
    """Scores so far apart that all but one probability vanish, and equal ones."""
    case = ref.Case([1, 2], [500, 70], 1, 128, 16, False, seed=9)
    for x in case.k:
        x *= 40.0
    _check(case, 4)
    case = ref.Case([1], [333], 1, 64, 16, False, seed=9)
    case.k[0].zero_()
    _check(case, 4)


def test_scale_and_strides():
    """A projection's [q | gate] per head read in place, keys and values out of one fused row."""
    case = ref.Case([2, 1], [40, 7], 2, 128, 16, True, seed=10)
    Hq, D = 6, 128
    q, z = _q(case, Hq, gate=True)
    qg = torch.cat([q, z], -1).cuda()
    kv = torch.zeros((sum(case.lens), 4 * D + 8), dtype=torch.bfloat16, device="cuda")
    kv[:, :2 * D] = torch.cat(case.k).cuda().view(-1, 2 * D)
    kv[:, 2 * D:4 * D] = torch.cat(case.v).cuda().view(-1, 2 * D)
    cache = case.empty_cache(runtime)
    cache.append(case.whole_batch(runtime), kv[:, :2 * D].view(-1, 2, D), kv[:, 2 * D:4 * D].view(-1, 2, D))
    got = cache.attend(case.device_batch(runtime), qg[..., :D], qg[..., D:], 0.07).cpu().double()
    want, spread = ref.attention(case, q, z, 0.07)
    assert ((got - want).abs() <= ref.attention_bound(want, spread)).all()


def test_quantised_vectors():
    """Scales at their limits: zero vectors, the least and largest magnitudes, exact powers, the
    448 border, infinities and NaN."""
    D = 64
    rows = torch.zeros((10, 1, D))
    rows[1] = 448.0
    rows[2] = 450.0
    rows[3, 0, 7] = 3.0e38
    rows[4, 0, 1] = 1e-40
    rows[5] = -2.0 ** -126
    rows[6] = torch.linspace(-5, 5, D)
    rows[7, 0, 0] = math.inf
    rows[8, 0, 9] = math.nan
    rows[9, 0, 0], rows[9, 0, 1] = 1.0, 2.0 ** -20
    x = rows.to(torch.bfloat16)
    case = ref.Case([10], [10], 1, D, 16, True, seed=0)
    case.k, case.v = [x], [-x]
    cache = case.filled_cache(runtime)
    k, v = (t.cpu().double() for t in cache.read(case.device_batch(runtime)))
    K, V = case.held()
    for got, want in ((k, K[0]), (v, V[0])):
        fine = [0, 1, 2, 3, 4, 5, 6, 9]
        assert torch.equal(got[fine], want[fine])
        assert torch.isnan(got[7:9]).all()
    b = cache.k_scales[int(case.table[0, 0]), 0].cpu().tolist()
    assert b[0] == 127 and b[1] == 127 and b[2] == 128 and b[4] == 10 and b[5] == 10 and b[7] == 255 and b[8] == 255


def test_bad_tables_and_lengths_are_reported():
    """Pages outside the pool read as zero and are not written; unusable lengths see nothing."""
    case = ref.Case([1, 1, 1], [40, 40, 20], 1, 64, 16, False, seed=11)
    cache = case.filled_cache(runtime)
    q, _ = _q(case, 2)
    b = case.device_batch(runtime)
    good = cache.attend(b, q.cuda())
    case.table[1, 1] = case.num_pages
    case.table[2, 0] = -1
    b = case.device_batch(runtime)
    got = cache.attend(b, q.cuda())
    assert int(cache.status.item()) == gdn.GDN_STATUS_PAGE_RANGE
    assert torch.equal(got[0], good[0]) and torch.isfinite(got).all()
    for kk in (case.k, case.v):
        kk[1][16:32] = 0
        kk[2][0:16] = 0
    want, spread = ref.attention(case, q)
    assert ((got.cpu().double() - want).abs() <= ref.attention_bound(want, spread)).all()
    before = cache.k_pages.clone()
    kv = torch.ones((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    case.table[0, 2] = 99999
    case.table[1, 2] = -5
    case.table[2, 1] = case.num_pages
    cache.append(case.device_batch(runtime), kv, kv)
    assert torch.equal(before.view(torch.int16), cache.k_pages.view(torch.int16))
    k, _ = cache.read(case.device_batch(runtime))
    assert (k == 0).all()
    cache.status.zero_()
    for lens in ([-1, 40, 20], [40, 1 << 30, 20]):
        case.lens = lens
        got = cache.attend(case.device_batch(runtime), q.cuda())
        assert int(cache.status.item()) & gdn.GDN_STATUS_BAD_SEQLENS
        assert (got[0 if lens[0] < 0 else 1] == 0).all()
        cache.status.zero_()


def test_graph_other_stream_and_reuse():
    """Captured in a graph on another stream, replayed after the cache and lengths changed."""
    case = ref.Case([1, 1], [300, 41], 2, 128, 16, True, seed=12)
    cache = case.filled_cache(runtime)
    q, _ = _q(case, 8)
    qd = q.cuda()
    b = case.device_batch(runtime)
    kv = torch.randn((2, 2, 128), device="cuda").to(torch.bfloat16)
    out = torch.empty_like(qd)
    ws = cache.workspace(8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        cache.append(b, kv, kv)
        cache.attend(b, qd, out=out, workspace=ws)
    torch.cuda.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cache.append(b, kv, kv)
        cache.attend(b, qd, out=out, workspace=ws)
    out.zero_()
    ws.fill_(0xff)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    b.tensors[1].copy_(torch.tensor([150, 41], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[1], first[1]) and not torch.equal(out[0], first[0])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("apart", [6, 17, 40])
def test_scales_far_apart(dim, apart):
    """Vectors of one head whose magnitudes differ by up to 2^apart, in and across key tiles, with
    the large values both seen strongly and not at all."""
    for new, length in ((1, 700), (40, 300)):
        case = ref.Case([new], [length], 1, dim, 32, True, seed=13)
        e = torch.randint(-apart, 1, (length, 1, 1), generator=torch.Generator().manual_seed(apart)).float()
        case.v[0] = (case.v[0].float() * torch.exp2(e)).to(torch.bfloat16)
        case.k[0] = (case.k[0].float() * torch.exp2((e / 8).round())).to(torch.bfloat16)
        _check(case, 4)
        case.v[0][::7] *= 2.0 ** 20
        case.k[0][::7] = 0
        _check(case, 4)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_nan_codes_past_the_end(dim):
    """What lies in a sequence's last page past its end may be anything, NaN codes among it."""
    for new, length in ((1, 45), (1, 130), (50, 170)):
        case = ref.Case([new], [length], 2, dim, 64, True, seed=14)
        cache = case.empty_cache(runtime)
        for p in (cache.k_pages, cache.v_pages):
            p.view(torch.uint8).fill_(0x7f)
        for s in (cache.k_scales, cache.v_scales):
            s.fill_(200)
        cache.append(case.whole_batch(runtime), torch.cat(case.k).cuda(), torch.cat(case.v).cuda())
        _check(case, 8, cache=cache)


@pytest.mark.parametrize("dim,quantised,heads,group,new", [
    (64, False, 8, 4, 1), (64, True, 8, 4, 1), (128, False, 4, 8, 1), (128, True, 4, 4, 1), (128, True, 4, 8, 2),
    (256, False, 2, 8, 1), (256, True, 4, 8, 1), (256, True, 4, 4, 3), (128, False, 4, 8, 40), (128, True, 4, 8, 40),
    (256, True, 2, 8, 40), (64, True, 4, 8, 40)])
def test_long_batches(dim, quantised, heads, group, new):
    """Enough cached positions that every CTA goes round its rings many times, several tiles each."""
    n, length = 48, 5000
    g = torch.Generator(device="cuda").manual_seed(15)
    page = 32
    per = -(-length // page)
    lens = [length - 37 * i for i in range(n)]
    k = torch.randn((n * length, heads, dim), generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn((n * length, heads, dim), generator=g, device="cuda").to(torch.bfloat16)
    cache = runtime.PagedKVCache(n * per, page, heads, dim, quantised)
    table = torch.randperm(n * per, generator=g, device="cuda").to(torch.int32).view(n, per)
    cu = torch.arange(0, n * length + 1, length, dtype=torch.int32, device="cuda")
    full = torch.full((n,), length, dtype=torch.int32, device="cuda")
    whole = runtime.KVBatch(cu, full, table, n * length, length)
    cache.append(whole, k, v)
    k, v = (x.view(n, length, heads, dim) for x in cache.read(whole))
    q = (torch.randn((n * new, heads * group, dim), generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    batch = runtime.KVBatch(torch.arange(0, n * new + 1, new, dtype=torch.int32, device="cuda"),
                            torch.tensor(lens, dtype=torch.int32, device="cuda"), table, n * new, new)
    got = cache.attend(batch, q).view(n, new, heads, group, dim).double()
    assert int(cache.status.item()) == 0
    q = q.view(n, new, heads, group, dim)
    for i in range(n):
        t = lens[i]
        s = torch.einsum("qhgd,jhd->hgqj", q[i].double(), k[i, :t].double()) / math.sqrt(dim)
        hide = torch.arange(t, device="cuda")[None] > torch.arange(t - new, t, device="cuda")[:, None]
        w = torch.softmax(s.masked_fill(hide, -math.inf), -1)
        want = torch.einsum("hgqj,jhd->qhgd", w, v[i, :t].double())
        spread = torch.einsum("hgqj,jhd->qhgd", w, v[i, :t].double().abs())
        assert ((got[i] - want).abs() <= ref.attention_bound(want, spread)).all(), i


@pytest.mark.parametrize("quantised", [False, True])
def test_pages_past_32_bit_offsets(quantised):
    """Pages whose elements lie more than 2^31 from the pool's start: the same bits as from a small
    pool, for a few rows and for many."""
    heads, dim, page = 8, 256, 256
    far = 2 ** 31 // (heads * dim * page)
    big = runtime.PagedKVCache(far + 6, page, heads, dim, quantised)
    small = runtime.PagedKVCache(8, page, heads, dim, quantised)
    g = torch.Generator(device="cuda").manual_seed(16)
    for new, length in ((1, 700), (40, 600)):
        kv = torch.randn((length, heads, dim), generator=g, device="cuda").to(torch.bfloat16)
        q = torch.randn((new, 2 * heads, dim), generator=g, device="cuda").to(torch.bfloat16)
        got = []
        for cache, pages in ((big, [far + 5, 1, far + 2]), (small, [6, 1, 3])):
            table = torch.tensor([pages], dtype=torch.int32, device="cuda")
            lens = torch.tensor([length], dtype=torch.int32, device="cuda")
            whole = runtime.KVBatch(torch.tensor([0, length], dtype=torch.int32, device="cuda"), lens, table, length, length)
            cache.append(whole, kv, kv)
            some = runtime.KVBatch(torch.tensor([0, new], dtype=torch.int32, device="cuda"), lens, table, new, new)
            got.append((*cache.read(whole), cache.attend(some, q)))
            assert int(cache.status.item()) == 0
        assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("dim,quantised", [(64, True), (128, False), (256, True)])
def test_many_short_pieces(dim, quantised):
    """More sequences than a CTA has threads, of a few tokens each; most have none."""
    new = [(5 if i % 7 == 3 else 0) for i in range(1500)]
    case = ref.Case(new, [n + i % 3 for i, n in enumerate(new)], 1, dim, 16, quantised, seed=17)
    _check(case, 8)


@pytest.mark.parametrize("new", [1, 2, 40])
def test_unknown_bound_on_new_tokens(new):
    """max_tokens 0: the same results within their bound as with it."""
    case = ref.Case([new, 1], [new + 400, 50], 2, 128, 32, False, seed=18)
    q, _ = _q(case, 8)
    want, spread = ref.attention(case, q)
    b = case.device_batch(runtime)
    free = runtime.KVBatch(*b.tensors, b.total_tokens)
    got = case.filled_cache(runtime).attend(free, q.cuda()).cpu().double()
    assert ((got - want).abs() <= ref.attention_bound(want, spread)).all()
