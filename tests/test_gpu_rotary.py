"""Rotary positions, and the cache's append with the heads' norm and rotation, against 64-bit forms.

Tolerances.  A turned element is two products and a sum of elements no larger than m = max(|a|, |b|) scale,
with sine and cosine to 2^-21 (2 units of f32 each, and the turn itself to 2^-25 of a radian's fraction):
2^-19 m, then the output's own half step.  With a norm, the mean's root and the two multiplications add four f32
roundings of the element: 2^-19 m holds them too."""
import math

import pytest
import torch

import mixer_ref as mr
import paged_ref as ref
from gated_deltanet_linear_09_gb300 import gdn, runtime

pytestmark = pytest.mark.gpu


def bound_of(want, size, dtype):
    return 2.0 ** -19 * size + mr.half_step(dtype) * (want.abs() + 2.0 ** -19 * size) + 1e-37


def pair_size(x, rot, scale, interleaved):
    """Largest of an element and its partner, times the scale; 0 for elements that stay."""
    s = torch.zeros_like(x)
    h = rot // 2
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :h], x[..., h:rot])
    m = (a.abs() + b.abs()) * abs(scale)
    if interleaved:
        s[..., 0:rot:2], s[..., 1:rot:2] = m, m
    else:
        s[..., :h], s[..., h:rot] = m, m
    return s


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [(1, 16, 2, 256, 64), (7, 3, 1, 128, 128), (33, 1, 0, 80, 40), (129, 2, 5, 81, 54),
                                           (5, 1, 1, 2, 2), (3, 2, 1, 1024, 1024), (300, 5, 2, 64, 8)])
def test_rotary(T, Hq, Hk, D, rot, dtype, interleaved):
    g = torch.Generator().manual_seed(T * D + rot)
    plan = runtime.Rotary(rot, base=1e6, interleaved=interleaved, scaling="bands", factor=4.0)
    row = torch.randn((T, (Hq + Hk) * D), generator=g).to(dtype)
    pos = torch.randint(-3000, 1 << 20, (T,), generator=g).to(torch.int32)
    dev = row.cuda()
    q, k = dev[:, :Hq * D].view(T, Hq, D), dev[:, Hq * D:].view(T, Hk, D) if Hk else None
    outs = plan.apply(pos.cuda(), q, k)
    assert (outs[1] is None) == (Hk == 0)
    for x, y in zip((q, k), outs):
        if x is None:
            continue
        x64 = x.cpu().double()
        want = mr.rotated(x64, pos, plan.frequencies, plan.scale, interleaved)
        mr.close(y, want, bound_of(want, pair_size(x64, rot, plan.scale, interleaved), dtype))
        assert torch.equal(y[..., rot:], x[..., rot:])


def test_far_positions_and_places():
    """Angles of positions to 2^31, where an f32 or an f64 product would be off."""
    f = [1.0, 0.7390851332151607, 1e-7, 2 * math.pi * 0.25]
    plan = runtime.Rotary.of(f)
    pos = torch.tensor([0, 1, -1, 2 ** 20, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32)
    x = torch.zeros((7, 1, 8))
    x[..., :4] = 1.0
    y = plan.apply(pos.cuda(), x.cuda())[0].cpu().double()
    from fractions import Fraction
    for i, p in enumerate(pos.tolist()):
        for j in range(4):
            turns = Fraction(int(plan.turns[j].item()) % 2 ** 64, 2 ** 64) * p % 1
            a = 2 * math.pi * float(turns)
            assert abs(y[i, 0, j] - math.cos(a)) < 2 ** -20 and abs(y[i, 0, j + 4] - math.sin(a)) < 2 ** -20
            # and the fraction is the frequency's, to what 53 bits of it leave
            assert abs(float(Fraction(int(plan.turns[j].item()) % 2 ** 64, 2 ** 64)) - f[j] / (2 * math.pi) % 1) < 2 ** -50


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rotary_in_place_strides_and_streams(dtype):
    """In place, over odd row and head distances, and on another stream: the bits of the plain call."""
    plan = runtime.Rotary(32, interleaved=False)
    base = torch.randn((40, 3, 77), device="cuda").to(dtype)
    x = base[..., 5:69]                                              # unaligned, head distance 77
    pos = torch.arange(40, dtype=torch.int32, device="cuda") * 1000
    want, _ = plan.apply(pos, x.contiguous())
    assert torch.equal(plan.apply(pos, x)[0], want)
    assert torch.equal(plan.apply(pos, None, x)[1], want)
    own = x.contiguous()
    assert plan.apply(pos, own, q_out=own)[0] is own and torch.equal(own, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = plan.apply(pos, x, stream=s)[0]
    s.synchronize()
    assert torch.equal(y, want)
    swapped = x.transpose(0, 1).contiguous().transpose(0, 1)         # heads outermost
    assert torch.equal(plan.apply(pos, swapped)[0], want)
    nothing = plan.apply(pos[:0], x[:0])[0]
    assert nothing.shape == (0, 3, 64)


def test_special_values():
    """Infinities and NaN stay in their pair."""
    plan = runtime.Rotary(16)
    x = torch.ones((2, 1, 32), device="cuda")
    x[0, 0, 3], x[1, 0, 20] = math.inf, math.nan
    y = plan.apply(torch.tensor([1, 2], dtype=torch.int32, device="cuda"), x)[0]
    bad = (~y.isfinite()).nonzero().tolist()
    assert bad == [[0, 0, 3], [0, 0, 11], [1, 0, 20]]


@pytest.mark.parametrize("rot", [20, 36, 10])
def test_vectors_of_all_sizes(rot):
    """Halves on 16-, 8- and 4-byte boundaries and on none: the bits of the plain call on a shifted copy."""
    plan = runtime.Rotary(rot)
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 777
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn((50, 3, 72), device="cuda").to(dtype)
        want = plan.apply(pos, x)[0]
        for shift, ld in ((1, 77), (2, 78), (4, 80), (8, 80)):
            wide = torch.zeros((50, 3, ld + 8), dtype=dtype, device="cuda")
            wide[..., shift:shift + 72] = x
            assert torch.equal(plan.apply(pos, wide[..., shift:shift + 72])[0], want)


def test_most_tokens():
    """Token counts at the end of 31 bits."""
    tokens = 2 ** 31 - 1
    plan = runtime.Rotary.of([math.pi / 2])
    pos = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    pos[-1] = 1
    x = torch.ones((tokens, 1, 2), dtype=torch.bfloat16, device="cuda")
    plan.apply(pos, x, q_out=x)
    assert x[-1, 0].tolist() == [-1.0, 1.0] and x[-2, 0].tolist() == [1.0, 1.0] and int((x[: 1 << 30] != 1.0).sum()) == 0


# ---------------------------------------------------------------- append with rotation

def case_inputs(case, Hq, seed, norm):
    g = torch.Generator().manual_seed(seed)
    T, H, D = case.tokens, case.heads, case.dim
    row = torch.randn((T, (2 * Hq + 2 * H) * D), generator=g).to(torch.bfloat16)
    w = [(0.2 * torch.randn(D, generator=g)).to(torch.bfloat16) if norm else None for _ in range(2)]
    q = row[:, :2 * Hq * D].view(T, Hq, 2 * D)[..., :D]
    k, v = (row[:, (2 * Hq + i * H) * D:(2 * Hq + (i + 1) * H) * D].view(T, H, D) for i in range(2))
    return row, q, k, v, w


def places(case):
    """Position of each packed token (None: no place)."""
    out = [None] * case.tokens
    for i, (a, t) in enumerate(zip(case.new, case.lens)):
        for r in range(a):
            p = t - a + r
            out[case.cu[i] + r] = p if p >= 0 and t > 0 else None
    return out


CASES = [([1] * 5, [1, 17, 300, 64, 33], 2, 128, 16, 128), ([40, 1, 0, 100, 7], [40, 500, 3, 131, 7], 1, 256, 64, 64),
         ([3, 20, 5], [3, 64, 2], 4, 64, 32, 48), ([257], [400], 2, 128, 128, 16), ([2000], [2000], 1, 64, 16, 64)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("new,lens,H,D,page,rot", CASES)
def test_append_rotated(new, lens, H, D, page, rot, norm, quantised, interleaved):
    Hq = 3 * H
    case = ref.Case(new, lens, H, D, page, quantised, seed=rot + H, pad_tokens=2)
    cache, b = case.empty_cache(runtime), case.device_batch(runtime)
    row, q, k, v, w = case_inputs(case, Hq, 11, norm)
    plan = runtime.Rotary(rot, base=1e4, interleaved=interleaved, scaling="bands", factor=8.0)
    dev = row.cuda()
    T = case.tokens
    qd = dev[:, :2 * Hq * D].view(T, Hq, 2 * D)[..., :D]
    kd, vd = (dev[:, (2 * Hq + i * H) * D:(2 * Hq + (i + 1) * H) * D].view(T, H, D) for i in range(2))
    wd = [None if x is None else x.cuda() for x in w]
    got_q = cache.append_rotated(b, plan, qd, kd, vd, q_norm=wd[0], k_norm=wd[1], weight_offset=1.0)
    got_k, got_v = cache.read(b)
    pos = places(case)
    live = torch.tensor([p is not None for p in pos])
    at = [p or 0 for p in pos]

    def whole(x, weight):
        x = x.double()
        if weight is not None:
            x = mr.rms(x, weight.double(), 1e-6, 1.0)
        y = mr.rotated(x, at, plan.frequencies, plan.scale, interleaved)
        size = x.abs() + pair_size(x, rot, plan.scale, interleaved)
        return y * live[:, None, None], size * live[:, None, None]
    want, size = whole(q, w[0])
    mr.close(got_q, want, bound_of(want, size, torch.bfloat16), "q")
    want, size = whole(k, w[1])
    if quantised:
        # one rounding to e4m3 in the vector's unit: half a step of the element, or of the least binade
        unit = torch.exp2(ref.scale_exponent(want * (1 + 2.0 ** -18)))[..., None]
        bound = 2.0 ** -19 * size + 2.0 ** -4 * (want.abs() + 2.0 ** -19 * size) + 2.0 ** -10 * unit
        mr.close(got_k, want, bound, "k")
        plain = case.empty_cache(runtime)                            # values are stored as by append()
        plain.append(b, kd, vd)
        assert torch.equal(plain.v_pages.view(torch.uint8), cache.v_pages.view(torch.uint8))
        assert torch.equal(plain.v_scales, cache.v_scales)
    else:
        mr.close(got_k, want, bound_of(want, size, torch.bfloat16), "k")
        assert torch.equal(got_v.cpu(), v * live[:, None, None])
    assert int(cache.status.item()) == (gdn.GDN_STATUS_BAD_SEQLENS if any(t < 0 for t in lens) else 0)


def test_without_rotation_or_norm_it_is_append():
    """Positions 0 everywhere and no norm: the pages of append(), the queries unchanged."""
    case = ref.Case([5, 30, 1], [9, 30, 200], 2, 128, 16, True, seed=3)
    _, q, k, v, _ = case_inputs(case, 4, 5, False)
    plan = runtime.Rotary(128)
    zero = torch.zeros(case.tokens, dtype=torch.int32, device="cuda")
    a, c, b = case.empty_cache(runtime), case.empty_cache(runtime), case.device_batch(runtime)
    q, k, v = (t.cuda().contiguous() for t in (q, k, v))
    a.append(b, k, v)
    got = c.append_rotated(b, plan, q, k, v, positions=zero)
    assert torch.equal(got, q)
    for x, y in ((a.k_pages, c.k_pages), (a.v_pages, c.v_pages), (a.k_scales, c.k_scales), (a.v_scales, c.v_scales)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert c.append_rotated(b, plan, None, k, v, positions=zero) is None


def test_given_positions_bad_pages_and_special_values():
    case = ref.Case([4, 3], [4, 20], 1, 64, 16, True, seed=8)
    _, q, k, v, _ = case_inputs(case, 2, 6, False)
    k = k.clone()
    k[0, 0, 5], k[5, 0, 60] = math.inf, math.nan
    case.table[0, 0] = 99                                            # outside the pool
    cache, b = case.empty_cache(runtime), case.device_batch(runtime)
    before = cache.k_pages.view(torch.uint8).clone()
    plan = runtime.Rotary(64)
    pos = torch.tensor([7, 7, 1, 0, -5, 100000, 3], dtype=torch.int32)
    got = cache.append_rotated(b, plan, q.cuda(), k.cuda(), v.cuda(), positions=pos.cuda())
    assert int(cache.status.item()) == gdn.GDN_STATUS_PAGE_RANGE
    assert bool((got[:4] == 0).all())
    want = mr.rotated(q.double(), pos, plan.frequencies)
    mr.close(got[4:], want[4:], bound_of(want, pair_size(q.double(), 64, 1.0, False), torch.bfloat16)[4:])
    kr, _ = cache.read(b)
    assert bool(kr[5].isnan().all()) and bool(kr[4].isfinite().all()) and bool(kr[6].isfinite().all())
    owned = {int(x) for x in case.table[1, :2]}
    for p in range(case.num_pages):
        if p not in owned:
            assert torch.equal(cache.k_pages.view(torch.uint8)[p], before[p])
