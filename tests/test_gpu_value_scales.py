"""Few query rows over an 8-bit cache whose value vectors' scales lie far apart: what a key adds
depends on its probability and its own scale, whatever the scales of the others are."""
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


def _faint_key(case, pos, size):
    """A key that queries with 8 in column 0 give no weight (a probability below 2^-200), with a
    value whose first elements are `size`."""
    case.k[0][:, :, 0] = 0
    case.k[0][pos] = 0
    case.k[0][pos, :, 0] = -400.0
    case.v[0][pos, :, :8] = size


def _queries(case, Hq, seed):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((case.tokens, Hq, case.dim), generator=g) * 1.5).to(torch.bfloat16)
    q[:, :, 0] = 8.0
    return q


@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 60, 2.0 ** 100, 3.0e38])
@pytest.mark.parametrize("dim,group", [(64, 4), (128, 4), (128, 12), (256, 8)])
def test_a_large_value_without_weight(dim, group, size):
    """At the start, the middle and the end of a sequence: the others' mean is left alone."""
    for length, pos in ((700, 0), (700, 333), (700, 640), (700, 699), (17, 3)):
        case = ref.Case([1], [length], 1, dim, 32, True, seed=31)
        q = _queries(case, group, 32)
        _faint_key(case, pos, size)
        got = case.filled_cache(runtime).attend(case.device_batch(runtime), q.cuda()).cpu().double()
        want, spread = ref.attention(case, q)
        assert ((got - want).abs() <= ref.attention_bound(want, spread)).all(), (length, pos)


def _repeated(case, n):
    """The case's one sequence n times, over the same pages: a batch in which a CTA walks many keys."""
    one, new = case.device_batch(runtime), case.new[0]
    cu = torch.arange(0, n * new + 1, new, dtype=torch.int32, device="cuda")
    return runtime.KVBatch(cu, one.tensors[1].repeat(n), one.tensors[2].repeat(n, 1), n * new, new)


@pytest.mark.parametrize("dim,group,new", [(64, 4, 4), (128, 4, 2), (128, 8, 2), (256, 4, 4)])
def test_a_large_value_hidden_from_earlier_tokens(dim, group, new):
    """The last token's value is as large as bf16 goes; the tokens before it do not see it."""
    n = 200
    for length in (new, 40, 1003):
        case = ref.Case([new], [length], 1, dim, 16, True, seed=33)
        q = _queries(case, group, 34)
        want, spread = ref.attention(case, q)
        case.v[0][length - 1] = 3.0e38
        got = case.filled_cache(runtime).attend(_repeated(case, n), q.repeat(n, 1, 1).cuda()).cpu().double()
        ok = (got.view(n, new, group, dim) - want).abs() <= ref.attention_bound(want, spread)
        assert ok[:, :new - 1].all(), length


@pytest.mark.parametrize("dim,group", [(64, 4), (128, 4), (128, 12), (256, 8)])
def test_small_probabilities_beside_a_large_value(dim, group):
    """In every warp's share of the keys: a faint key whose value is 2^17 times the others', a strong key
    without a value, and hundreds of keys of one small probability that carry the result.  A query of its
    own for each of the sequences: probabilities from 2^-9 to 2^-11."""
    length, n = 4096, 150
    case = ref.Case([1], [length], 2, dim, 32, True, seed=35)
    g = torch.Generator().manual_seed(36)
    case.k[0].zero_()
    case.v[0] = (1.0 + 0.2 * torch.randn((length, 2, dim), generator=g)).to(torch.bfloat16)
    at = (torch.arange(0, length, 512)[:, None] + torch.arange(0, 128, 16)[None]).flatten()
    case.k[0][at, :, 0] = 10 * math.log(2.0) * math.sqrt(dim) / 8.0
    case.v[0][at] = 0
    case.k[0][at + 1, :, 0] = -400.0
    case.v[0][at + 1] = 2.0 ** 17
    q = torch.zeros((n, 2 * group, dim), dtype=torch.bfloat16)
    q[:, :, 0] = (7.2 + 1.6 * torch.arange(n)[:, None] / n).to(torch.bfloat16)
    got = case.filled_cache(runtime).attend(_repeated(case, n), q.cuda()).cpu().double()
    K, V = (x[0] for x in case.held())
    score = q[:, 0, 0].double()[:, None] * K[None, :, 0, 0] / math.sqrt(dim)
    want = (torch.softmax(score, 1) @ V.reshape(length, -1)).view(n, 2, 1, dim).expand(n, 2, group, dim).reshape(n, -1, dim)
    assert ((got - want).abs() <= ref.attention_bound(want, want)).all()      # (no value is negative)
