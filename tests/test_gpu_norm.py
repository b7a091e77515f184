"""gdn_rms_norm against its formula in 64 bits: both activation types, widths on and off the
vector grid, every output kind, strides, in-place sums, zero and non-finite rows."""
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


def _formula(x, r, w, offset, eps):
    h = x.double() if r is None else x.double() + r.double()
    return h, h / torch.sqrt((h ** 2).mean(1, keepdim=True) + eps) * (w.double() + offset)


WIDTHS = [1, 7, 8, 64, 100, 128, 250, 1000, 1024, 2047, 2048, 2056, 4096, 5120, 8191, 8200, 16384, 32768]


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", WIDTHS)
def test_norm(n, act):
    g = torch.Generator().manual_seed(n)
    rows = 5 if n > 2000 else 37
    x = torch.randn((rows, n), generator=g).to(act)
    r = (torch.randn((rows, n), generator=g) * 3).to(act)
    w = (torch.randn((n,), generator=g) * 0.1).to(act)
    x[1].zero_()
    r[1].zero_()
    half = torch.finfo(act).eps / 2
    # f32: the sum of n squares, the root and two products, each within a few roundings
    f32 = (8 + math.sqrt(n)) * 2.0 ** -24
    for res, offset in ((r, 1.0), (None, 0.0)):
        h, want = _formula(x, res, w, offset, 1e-6)
        for quant in ("none", "row", "block"):
            y, scales, total = runtime.rms_norm(x.cuda(), w.cuda(), None if res is None else res.cuda(),
                                                weight_offset=offset, quant=quant)
            if res is not None:
                assert ((total.cpu().double() - h).abs() <= half * h.abs()).all()
            if quant == "none":
                # the sum x + r is itself rounded to f32 before the norm
                assert ((y.cpu().double() - want).abs() <= (half + f32 + 2.0 ** -23) * want.abs() + 1e-30).all()
                continue
            size = n if quant == "row" else 128
            for c in range(0, n, size):
                part = want[:, c:c + size]
                s = (part.abs().amax(1) / 448.0).clamp(min=2.0 ** -120)
                got_s = scales[:, c // size].cpu().double()
                assert ((got_s - s).abs() <= (f32 + 2.0 ** -22) * s).all()
                got = y[:, c:c + size].cpu().double() * got_s[:, None]
                # half an e4m3 step of the value (2^-4), or of the least normal in scaled units
                bound = (2.0 ** -4 + 2.0 ** -18) * part.abs() + 2.0 ** -10 * got_s[:, None] * (1 + 2.0 ** -18)
                assert ((got - part).abs() <= bound).all()
            assert (y[1].cpu().float() == 0).all()


def test_strides_and_in_place():
    g = torch.Generator().manual_seed(3)
    buf = torch.randn((9, 700), generator=g).to(torch.bfloat16).cuda()
    res = torch.randn((9, 640), generator=g).to(torch.bfloat16).cuda()
    w = torch.randn((640,), generator=g).to(torch.bfloat16).cuda()
    x = buf[:, :640]
    h, want = _formula(x.cpu(), res.cpu(), w.cpu(), 0.0, 1e-5)
    y = torch.empty((9, 640), dtype=torch.bfloat16, device="cuda")
    gdn.gdn_rms_norm(x, w, y, res, res, eps=1e-5)          # the sum replaces the residual
    assert ((y.cpu().double() - want).abs() <= 2.0 ** -7.9 * want.abs()).all()
    assert ((res.cpu().double() - h).abs() <= 2.0 ** -8 * h.abs()).all()


def test_non_finite_rows_stay_in_their_rows_and_groups():
    x = torch.randn((6, 512)).to(torch.bfloat16)
    x[1, 5] = math.nan
    x[3, 300] = math.inf
    w = torch.ones((512,), dtype=torch.bfloat16)
    y, s, _ = runtime.rms_norm(x.cuda(), w.cuda(), quant="block")
    y, s = y.float().cpu(), s.cpu()
    assert torch.isnan(y[1]).all() and torch.isnan(s[1]).all()
    assert torch.isnan(s[3, 2]) and torch.isfinite(s[3, [0, 1, 3]]).all()
    for r in (0, 2, 4, 5):
        assert torch.isfinite(y[r]).all() and torch.isfinite(s[r]).all()
    y, s, _ = runtime.rms_norm(x.cuda(), w.cuda(), quant="row")
    assert torch.isnan(s[1, 0]) and torch.isnan(s[3, 0]) and torch.isfinite(s[[0, 2, 4, 5], 0]).all()


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    y, _, _ = runtime.rms_norm(x, torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    assert y.shape == (0, 64)


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [2, 33, 129, 130, 254, 255, 258, 511, 514, 1022, 1023, 1026, 2046, 4098, 8190, 16382, 20001, 32766])
def test_norm_off_the_vector_grid(n, act):
    test_norm(n, act)


@pytest.mark.parametrize("n", [300, 301, 1300, 2051])
def test_non_finite_groups_off_the_vector_grid(n):
    x = torch.randn((4, n)).to(torch.bfloat16)
    x[2, 130] = math.inf                           # its row's norm is zero elsewhere, NaN there
    x[1, 7] = math.nan
    y, s, _ = runtime.rms_norm(x.cuda(), torch.ones((n,), dtype=torch.bfloat16).cuda(), quant="block")
    y, s = y.float().cpu(), s.cpu()
    assert torch.isnan(s[1]).all() and torch.isnan(y[1]).all()
    assert torch.isnan(s[2, 1]) and torch.isfinite(s[2, 0]) and torch.isfinite(s[2, 2:]).all()
    assert torch.isfinite(s[[0, 3]]).all() and torch.isfinite(y[[0, 3]]).all()
