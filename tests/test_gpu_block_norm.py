"""The norms around a block with its gate and residual scale, against the 64-bit form.

Tolerances.  total: the block's term b (norm, gate, scales) is some ten f32 roundings and, for bf16, a
sigmoid off by 2^-20: 2^-18 of |b| for f32, 2^-17 for bf16; the sum and the output add half a step each.  y adds the
same for its norm, whose mean takes the errors of total's terms."""
import math

import pytest
import torch

import mixer_ref as mr
from gated_deltanet_linear_09_gb300 import gdn, runtime
from gpu_util import Guarded

pytestmark = pytest.mark.gpu


def make(rows, n, group, dtype, seed, **have):
    g = torch.Generator().manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=g).to(dtype)
    t = dict(x=rand(rows, n))
    if have.get("gate", True):
        t["gate"] = rand(rows, n) * 3
    if have.get("residual", True):
        t["residual"] = rand(rows, n) * 4
    if have.get("post", True):
        t["post"] = rand(group) * 0.2
    if have.get("pre", True):
        t["pre"] = rand(n) * 0.2
    if have.get("channel", True):
        t["channel_scale"] = rand(n) * 0.5
    return t


def check(t, dtype, got, gate_act="sigmoid", scale=1.0, offset=1.0):
    d = {k: v.double() for k, v in t.items()}
    if "channel_scale" in d:
        d["channel"] = d.pop("channel_scale")
    h, y = mr.block(gate_act=gate_act, scale=scale, offset=offset, **d)
    rel = 2.0 ** (-17 if dtype == torch.bfloat16 else -18)
    half = mr.half_step(dtype)
    b = (h - d.get("residual", 0.0)).abs()
    off = rel * b + 2.0 ** -24 * h.abs()
    mr.close(got[0], h, off + half * (h.abs() + off) + 1e-37, "total")
    assert (got[1] is None) == (y is None)
    if y is not None:
        # an element's own error, and the row's mean's
        inv = y.abs() / h.abs().clamp(min=1e-30)
        row = (off * off).mean(-1, keepdim=True).sqrt() / (h * h).mean(-1, keepdim=True).sqrt().clamp(min=1e-30)
        err = off * inv + y.abs() * (row + 2.0 ** -20)
        mr.close(got[1], y, err + half * (y.abs() + err) + 1e-37, "y")


def run(t, **kw):
    return runtime.block_norm(**{k: v.cuda() for k, v in t.items()}, weight_offset=1.0, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n", [(1, 5120), (3, 1), (5, 7), (2, 129), (4, 256), (7, 512), (3, 1000), (2, 2047), (3, 4096),
                                    (2, 6144), (3, 8192), (2, 8191), (2, 16384), (1, 32768), (1, 32767), (300, 64)])
def test_rows(rows, n, dtype):
    for act in ("sigmoid", "silu"):
        t = make(rows, n, n, dtype, rows + n)
        check(t, dtype, run(t, gate_act=act, scale=0.5), act, 0.5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("heads", [1, 2, 3, 40, 100])
def test_groups(heads, group, dtype):
    t = make(5, heads * group, group, dtype, heads + group)
    check(t, dtype, run(t, gate_act="silu"), "silu")


@pytest.mark.parametrize("missing", [("gate",), ("residual",), ("post",), ("pre",), ("channel",), ("gate", "post", "channel"),
                                     ("residual", "pre"), ("gate", "residual", "post", "channel")])
def test_parts(missing):
    for n in (256, 255):
        t = make(6, n, n, torch.bfloat16, n, **{m: False for m in missing})
        check(t, torch.bfloat16, run(t))


def test_strides_guards_and_in_place():
    n = 640
    for dtype in (torch.bfloat16, torch.float32):
        for ld in (n + 8, n + 3):
            t = make(9, n, 64 if ld % 8 == 0 else n, dtype, ld)
            wide = {k: torch.zeros((9, ld), dtype=dtype).cuda() for k in ("x", "gate", "residual")}
            for k, w in wide.items():
                w[:, :n] = t[k].cuda()
            total, y = Guarded((9, n), dtype), Guarded((9, n), dtype)
            got = runtime.block_norm(**{k: v.cuda() for k, v in t.items() if k not in wide},
                                     **{k: w[:, :n] for k, w in wide.items()}, weight_offset=1.0, total=total.view, y=y.view)
            total.check()
            y.check()
            check(t, dtype, got)
        t = make(9, n, n, dtype, 1)
        want = run(t)
        r = t["residual"].cuda()
        got = runtime.block_norm(**{k: v.cuda() for k, v in t.items() if k != "residual"}, residual=r, total=r, weight_offset=1.0)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0] is r


def test_special_values_and_graph():
    t = make(4, 512, 128, torch.bfloat16, 2)
    t["x"][1, 130] = math.nan
    t["residual"][2, 5] = math.inf
    t["gate"][3, 7] = -math.inf
    t["x"][0] = 0
    got = run(t)
    assert torch.equal((~got[0][1].isfinite()).nonzero().flatten().cpu(), torch.arange(128, 256))
    assert bool(got[1][1].isnan().all()) and bool(got[0][0].isfinite().all())
    assert float(got[0][2, 5]) == math.inf and float(got[0][3, 7]) == float(t["residual"][3, 7])
    x = {k: v.cuda() for k, v in t.items()}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = runtime.block_norm(**x, weight_offset=1.0)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, got):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert runtime.block_norm(x["x"][:0])[0].shape == (0, 512)
    assert gdn.GDN_GATE_SILU == 2


@pytest.mark.parametrize("dtype,rows,n,pad", [
    (torch.bfloat16, 20000, 264, 0), (torch.bfloat16, 5000, 1600, 8), (torch.bfloat16, 1300, 12296, 0),     # aligned rows
    (torch.bfloat16, 20001, 129, 0), (torch.bfloat16, 20000, 130, 2), (torch.bfloat16, 7001, 1001, 2),       # pairs
    (torch.bfloat16, 3001, 4097, 4), (torch.bfloat16, 1301, 8191, 0), (torch.bfloat16, 611, 15001, 0),
    (torch.bfloat16, 20001, 131, 1), (torch.bfloat16, 7001, 1002, 1), (torch.bfloat16, 650, 20001, 1),       # anywhere
    (torch.float32, 20001, 257, 0), (torch.float32, 4001, 1500, 4), (torch.float32, 1301, 7001, 0),
    (torch.float32, 1301, 8192, 0), (torch.float32, 620, 12289, 3)])
def test_many_rows(dtype, rows, n, pad):
    """Rows enough for CTAs that stay, on and off the boundaries, with NaN between them."""
    t = make(rows, n, n, dtype, rows + n)
    dev = {k: v.cuda() for k, v in t.items()}
    for k in ("x", "gate", "residual"):
        wide = torch.full((rows, n + pad), math.nan, dtype=dtype, device="cuda")
        wide[:, :n] = dev[k]
        dev[k] = wide[:, :n]
    total, y = Guarded((rows, n), dtype), Guarded((rows, n), dtype)
    got = runtime.block_norm(**dev, weight_offset=1.0, gate_act="silu", scale=0.5, total=total.view, y=y.view)
    total.check()
    y.check()
    check({k: v.cuda() for k, v in t.items()}, dtype, got, "silu", 0.5)
    # parts of it, in place of the residual
    dense = t["residual"].cuda()
    alone, _ = runtime.block_norm(dev["x"], dev["post"], residual=dense.clone(), weight_offset=1.0)
    runtime.block_norm(dev["x"], dev["post"], residual=dense, total=dense, weight_offset=1.0)
    assert torch.equal(alone, dense)
    check({k: t[k].cuda() for k in ("x", "post", "residual")}, dtype, (dense, None))
    # its last rows by themselves
    few = runtime.block_norm(**{k: v[-3:].clone() if k in ("x", "gate", "residual") else v for k, v in dev.items()},
                             weight_offset=1.0, gate_act="silu", scale=0.5)
    check({k: (v[-3:] if k in ("x", "gate", "residual") else v).cuda() for k, v in t.items()}, dtype, few, "silu", 0.5)


def test_most_rows():
    """Row counts at the end of 31 bits."""
    rows = 2 ** 31 - 1
    x = torch.ones((rows, 1), dtype=torch.bfloat16, device="cuda")
    x[-1], x[-2] = 3.0, -5.0
    total, _ = runtime.block_norm(x, scale=2.0)
    assert total[-1].item() == 6.0 and total[-2].item() == -10.0 and total[0].item() == 2.0
    assert int((total[: 1 << 30] != 2.0).sum()) == 0
