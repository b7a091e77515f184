"""What a row does not see changes no bit of its result: later tokens' keys and values, and what the
pages hold past a sequence's end."""
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


def _cache(case, garbage):
    """The case's sequences in pages that held `garbage` before: a number, or codes and scale bytes."""
    c = case.empty_cache(runtime)
    for p in (c.k_pages, c.v_pages):
        if case.quantised:
            p.view(torch.uint8).fill_(garbage[0])
        else:
            p.fill_(garbage)
    for s in (c.k_scales, c.v_scales):
        if s is not None:
            s.fill_(garbage[1])
    c.append(case.whole_batch(runtime), torch.cat(case.k).cuda(), torch.cat(case.v).cuda())
    return c


SHAPES = [  # dim, quantised, group, new tokens: few rows, one block and two blocks of many
    (64, False, 4, 4), (64, True, 4, 4), (128, False, 4, 2), (128, False, 2, 7), (128, True, 4, 4), (256, False, 4, 3),
    (256, True, 8, 2), (64, False, 4, 20), (64, True, 4, 20), (128, False, 4, 30), (128, True, 4, 30),
    (256, False, 4, 30), (256, True, 4, 30), (128, False, 8, 40), (128, True, 8, 40),
]


@pytest.mark.parametrize("dim,quantised,group,new", SHAPES)
def test_later_tokens_change_no_bit(dim, quantised, group, new):
    for seed, length in ((41, new), (42, new + 13), (43, 300)):
        case = ref.Case([new], [length], 2, dim, 16, quantised, seed=seed)
        case.k[0] = (case.k[0].float() * 3).to(torch.bfloat16)
        g = torch.Generator().manual_seed(seed)
        q = (torch.randn((new, 2 * group, dim), generator=g) * 1.5).to(torch.bfloat16).cuda()
        rows, k0 = None, case.k[0].clone()
        v0 = case.v[0].clone()
        for k, v in ((None, None), (50.0, 0.0), (-3.0, 1e30), (0.0, 3e38), (math.nan, math.nan), (1.0, math.inf),
                     (math.inf, -math.inf)):
            case.k[0], case.v[0] = k0.clone(), v0.clone()
            if k is not None:
                case.k[0][-1] = case.k[0][-1] * k if math.isfinite(k) and k else k
                case.v[0][-1] = v
            got = case.filled_cache(runtime).attend(case.device_batch(runtime), q)[:new - 1].view(torch.int16)
            rows = got if rows is None else rows
            assert torch.equal(got, rows), (length, k, v)


@pytest.mark.parametrize("dim,quantised,group,new", SHAPES)
def test_bytes_past_the_end_change_no_bit(dim, quantised, group, new):
    """Among many sequences, every other one a token shorter, so that tiles have rows that hold nothing."""
    n = 400
    counts = [new - i % 2 for i in range(n)]
    case = ref.Case(counts, [a + 3 + i % 29 for i, a in enumerate(counts)], 2, dim, 16, quantised, seed=44)
    g = torch.Generator().manual_seed(45)
    q = (torch.randn((case.tokens, 2 * group, dim), generator=g) * 4).to(torch.bfloat16).cuda()
    b = case.device_batch(runtime)
    fills = ((0, 127), (0x7f, 255), (0x7e, 247), (0xfe, 200), (0x38, 10)) if quantised else (0.0, math.nan, 3e38, -1e20, math.inf)
    outs = [_cache(case, x).attend(b, q).view(torch.int16) for x in fills]
    for x, out in zip(fills, outs):
        assert torch.equal(out, outs[0]), x


@pytest.mark.parametrize("dim,group,new", [(64, 2, 4), (128, 4, 3), (256, 2, 6), (64, 4, 12), (128, 2, 60), (128, 8, 40), (256, 4, 50)])
def test_infinite_values_reach_the_rows_that_see_them(dim, group, new):
    """In a bf16 cache: a row that sees +inf in a column has it there, one that sees both has NaN."""
    case = ref.Case([new], [new + 30], 1, dim, 16, False, seed=46)
    g = torch.Generator().manual_seed(47)
    q = torch.randn((new, group, dim), generator=g).to(torch.bfloat16)
    last = new + 29
    case.v[0][last - 2, 0, 3] = math.inf
    case.v[0][last - 2, 0, 7] = -math.inf
    case.v[0][last - 1, 0, 9] = math.inf
    case.v[0][last, 0, 9] = -math.inf
    case.v[0][last - 1, 0, 20] = math.nan
    case.v[0][last, 0, 20] = math.inf
    got = case.filled_cache(runtime).attend(case.device_batch(runtime), q.cuda()).cpu().double()
    want, spread = ref.attention(case, q)
    want[:new - 3][want[:new - 3] != want[:new - 3]] = 0      # 0 * inf of keys past a row's own
    bound = ref.attention_bound(want, spread)
    for t in range(new):
        for col, places in ((3, {last - 2: math.inf}), (7, {last - 2: -math.inf}),
                            (9, {last - 1: math.inf, last: -math.inf}), (20, {last - 1: math.nan, last: math.inf})):
            seen = [x for p, x in places.items() if p <= t + 30]
            if not seen:
                assert torch.isfinite(got[t, :, col]).all(), (t, col)
            elif len(set(seen)) > 1 or math.isnan(seen[0]):
                assert torch.isnan(got[t, :, col]).all(), (t, col)
            else:
                assert (got[t, :, col] == seen[0]).all(), (t, col)
    cols = [d for d in range(dim) if d not in (3, 7, 9, 20)]
    assert ((got - want).abs() <= bound)[:, :, cols].all()
