"""Plain 64-bit forms of the norm, cache and attention operators, and batches to test them on."""
from __future__ import annotations

import math

import torch

E4M3 = torch.float8_e4m3fn


def e4m3_round(x):
    """Nearest e4m3 value (ties to even) of a float64 tensor with |x| <= 448."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.sign(x) * torch.round(a / step) * step


def scale_exponent(x):
    """[..., D] float64 -> the least e >= -117 with max|x| <= 448 * 2^e, 0 for a zero vector."""
    amax = x.abs().amax(-1)
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / 448.0))
    e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= 448.0 * torch.exp2(e - 1), e - 1, e)
    return torch.where(amax > 0, e, torch.zeros_like(e)).clamp(min=-117.0)


class Case:
    """A ragged batch over a shuffled page pool: new[i] new tokens of sequence i, lens[i] cached
    positions including them.  Pages that no sequence owns, and the rest of partly used ones, hold
    garbage (NaN in a bf16 cache, NaN scales in an 8-bit one)."""

    def __init__(self, new, lens, heads, dim, page, quantised, seed=0, pad_tokens=0, table_extra=1):
        g = torch.Generator().manual_seed(seed)
        self.new, self.lens, self.heads, self.dim, self.page = list(new), list(lens), heads, dim, page
        self.quantised = quantised
        n = len(new)
        counts = [-(-max(0, t) // page) for t in lens]
        self.num_pages = sum(counts) + 2
        order = torch.randperm(self.num_pages, generator=g).tolist()
        width = max(counts + [1]) + table_extra
        table = torch.full((n, width), -7, dtype=torch.int32)      # entries that must not be read
        at = 0
        for i, c in enumerate(counts):
            table[i, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
            at += c
        self.table = table
        self.cu = [0]
        for x in new:
            self.cu.append(self.cu[-1] + x)
        self.tokens = self.cu[-1] + pad_tokens
        # what the sequences hold, in bf16
        self.k = [torch.randn((max(0, t), heads, dim), generator=g).to(torch.bfloat16) for t in lens]
        self.v = [torch.randn((max(0, t), heads, dim), generator=g).to(torch.bfloat16) for t in lens]

    def device_batch(self, runtime):
        dev = "cuda"
        cu = torch.tensor(self.cu, dtype=torch.int32, device=dev)
        lens = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        return runtime.KVBatch(cu, lens, self.table.to(dev), self.tokens, max(self.new + [0]))

    def whole_batch(self, runtime):
        """The same sequences with every cached position as a token."""
        dev = "cuda"
        cu = [0]
        for t in self.lens:
            cu.append(cu[-1] + max(0, t))
        return runtime.KVBatch(torch.tensor(cu, dtype=torch.int32, device=dev),
                               torch.tensor([max(0, t) for t in self.lens], dtype=torch.int32, device=dev),
                               self.table.to(dev), cu[-1], max(self.lens + [0]))

    def empty_cache(self, runtime):
        c = runtime.PagedKVCache(self.num_pages, self.page, self.heads, self.dim, self.quantised)
        if self.quantised:
            for p in (c.k_pages, c.v_pages):
                p.view(torch.uint8).fill_(0x7b)
            for s in (c.k_scales, c.v_scales):
                s.fill_(255)
        else:
            c.k_pages.fill_(math.nan)
            c.v_pages.fill_(math.nan)
        return c

    def filled_cache(self, runtime):
        """A cache holding the sequences (through the library's append) and what it stands for."""
        c = self.empty_cache(runtime)
        b = self.whole_batch(runtime)
        if b.total_tokens:
            c.append(b, torch.cat(self.k).cuda(), torch.cat(self.v).cuda())
        return c

    def held(self):
        """The values the cache holds, float64 per sequence."""
        out = []
        for xs in (self.k, self.v):
            ys = []
            for x in xs:
                x = x.double()
                if self.quantised and x.numel():
                    s = torch.exp2(scale_exponent(x))[..., None]
                    x = e4m3_round(x / s) * s
                ys.append(x)
            out.append(ys)
        return out


def attention(case, q, gate=None, scale=None):
    """float64 (out, spread): spread = sum_j p_j |v_j|, what rounding the probabilities scales with."""
    K, V = case.held()
    T, Hq, D = q.shape
    g = Hq // case.heads
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = torch.zeros((T, Hq, D), dtype=torch.float64)
    spread = torch.zeros_like(out)
    for i, (a, t) in enumerate(zip(case.new, case.lens)):
        for r in range(a):
            p = t - a + r
            row = case.cu[i] + r
            if p < 0 or t <= 0:
                continue
            qq = q[row].double().view(case.heads, g, D)
            s = torch.einsum("hgd,jhd->hgj", qq, K[i][:p + 1]) * scale
            w = torch.softmax(s, -1)
            out[row] = torch.einsum("hgj,jhd->hgd", w, V[i][:p + 1]).reshape(Hq, D)
            spread[row] = torch.einsum("hgj,jhd->hgd", w, V[i][:p + 1].abs()).reshape(Hq, D)
    if gate is not None:
        z = torch.sigmoid(gate.double())
        out, spread = out * z, spread * z
    return out, spread


def attention_bound(out, spread):
    """Probabilities rounded to bf16 (half a step, 2^-8, of each), the output's own rounding
    (2^-8), and 2^-10 for f32 sums, scores and exponentials."""
    return (2.0 ** -8 + 2.0 ** -10) * spread + 2.0 ** -8 * out.abs() + 1e-30
