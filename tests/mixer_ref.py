"""Plain 64-bit forms of the operators between a layer's projections."""
from __future__ import annotations

import math

import torch

BF16 = 2.0 ** -8       # half a step of bf16, relative
F32 = 2.0 ** -24


def half_step(dtype):
    return BF16 if dtype == torch.bfloat16 else F32


def rotated(x, pos, freq, scale=1.0, interleaved=False):
    """x [T][heads][D] float64, pos [T] int64, freq [R / 2]."""
    T = x.shape[0]
    h = len(freq)
    y = x.clone()
    for i, f in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        # the angle modulo a turn, by whole numbers where 53 bits would not do
        t = torch.tensor([math.remainder(int(p) * f, 2 * math.pi) for p in pos], dtype=torch.float64)
        c, s = torch.cos(t)[:, None] * scale, torch.sin(t)[:, None] * scale
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y.view(T, *x.shape[1:])


def rms(x, w, eps, offset):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (offset + w)


def block(x, post=None, gate=None, gate_act="sigmoid", scale=1.0, channel=None, residual=None, pre=None, eps=1e-6,
          offset=0.0):
    b = x
    if post is not None:
        g = post.shape[0]
        b = rms(b.view(b.shape[0], -1, g), post, eps, offset).reshape(x.shape)
    if gate is not None:
        s = torch.sigmoid(gate)
        b = b * (gate * s if gate_act == "silu" else s)
    if channel is not None:
        b = b * channel
    h = scale * b + (residual if residual is not None else 0.0)
    return h, None if pre is None else rms(h, pre, eps, offset)


def decay(S, q, k, v, g, scale=None):
    """One sequence token by token: S [Hv][dk][dv], q, k [T][Hk][dk], v [T][Hv][dv], g [Hv] or [T][Hv], all
    float64 -> (out [T][Hv][dv], state, size): size = scale sum |q||S|, what roundings of S and of the scores
    scale with."""
    T, Hv, dv = v.shape
    rep = Hv // q.shape[1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    g = g.expand(T, Hv)
    S = S.clone()
    M = S.abs()
    out, size = torch.zeros_like(v), torch.zeros_like(v)
    for t in range(T):
        e = torch.exp(g[t])[:, None, None]
        S = torch.where(e == 0, torch.zeros_like(S), e * S) + k[t][:, :, None] * v[t][:, None, :]
        M = torch.where(e == 0, torch.zeros_like(M), e * M) + (k[t][:, :, None] * v[t][:, None, :]).abs()
        out[t] = scale * torch.einsum("hkv,hk->hv", S, q[t])
        size[t] = scale * torch.einsum("hkv,hk->hv", M, q[t].abs())
    return out, S, size, M


def close(got, want, bound, what=""):
    """|got - want| <= bound where want is finite; the same infinities and NaN elsewhere."""
    got, want, bound = got.detach().cpu().double(), want.cpu(), bound.cpu()
    fine = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), f"{what}: infinities"
    excess = ((got - want).abs() - bound)[fine]
    assert excess.numel() == 0 or float(excess.max()) <= 0, f"{what}: over the bound by {float(excess.max()):.3e}"
