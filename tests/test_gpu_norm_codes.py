"""The 8-bit codes of gdn_rms_norm are those of y / scale: values beside the halfway points of two codes."""
import pytest
import torch

from gated_deltanet_linear_09_gb300 import gdn, runtime

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from gated_deltanet_linear_09_gb300 import build
    build.build()
    gdn.load()


def _halfway():
    codes = torch.arange(127, dtype=torch.uint8).view(E4M3).double()       # 0 to 448
    return (codes[1:] + codes[:-1]) / 2


def _weights(top, n, seed):
    """f32 weights whose largest is `top`; the others lie within a few units of halfway between codes."""
    scale = torch.tensor(top, dtype=torch.float32) / 448
    g = torch.Generator().manual_seed(seed)
    h = _halfway()
    w = (h[torch.randint(0, len(h), (n,), generator=g)] * scale.double()).float()
    w = (w.view(torch.int32) + torch.randint(-3, 4, (n,), generator=g, dtype=torch.int32)).view(torch.float32)
    w *= torch.randint(0, 2, (n,), generator=g) * 2 - 1
    w[::128] = top
    return w, scale


@pytest.mark.parametrize("quant", ["row", "block"])
@pytest.mark.parametrize("n", [512, 2048, 16384])
def test_codes_beside_halfway_points(n, quant):
    """Rows of +-1 have the norm 1, so y is the weight and nothing but the quotient is rounded."""
    x = (torch.randint(0, 2, (3, n), generator=torch.Generator().manual_seed(1)) * 2 - 1).float()
    for seed, top in enumerate((1.0, 0.3, 1.7, 3.1415927, 447.9, 1e-3, 5.5e4, 1e-20, 2e25)):
        w, scale = _weights(top, n, seed)
        y, s, _ = runtime.rms_norm(x.cuda(), w.cuda(), eps=0.0, quant=quant)
        assert (s.cpu() == scale).all(), top
        want = (x * (w / scale)).to(E4M3)
        assert torch.equal(y.cpu().view(torch.uint8), want.view(torch.uint8)), top


def test_infinities_and_nan():
    """A group with an infinity has an infinite scale, zeros and a NaN; one with a NaN is NaN."""
    for n in (256, 2047, 4096):
        w = torch.ones(n)
        w[3], w[130] = torch.inf, torch.nan
        y, s, _ = runtime.rms_norm(torch.ones((2, n), device="cuda"), w.cuda(), eps=0.0, quant="block")
        s, y = s.cpu(), y.cpu().float()
        assert (s[:, 0] == torch.inf).all() and s[:, 1].isnan().all()
        assert y[:, 3].isnan().all() and (y[:, :3] == 0).all() and (y[:, 4:128] == 0).all() and y[:, 128:min(n, 256)].isnan().all()
