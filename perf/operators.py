"""Timed cases of the operators around the hybrid models' full-attention layers: the residual
RMSNorm (bf16, f32 and scaled 8-bit outputs), the paged key/value cache (quantised as it is
written, read back), and attention of new tokens over that cache (one token per sequence up to
whole prompts).  ``own`` selects the library's kernels; otherwise the same results are computed
by elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token's hidden state entering a layer: launch latency is all there is
        dict(name="norm_token", op="norm", rows=1, n=5120, act="bf16", residual=True, quant="none",
             offset=1.0),
        # f32 activations of an odd width, no residual: unaligned rows
        dict(name="norm_odd_f32", op="norm", rows=1537, n=2047, act="f32", residual=False,
             quant="none", offset=0.0),
        # a prompt batch entering an 8-bit projection: one scale per 128 columns
        dict(name="norm_prompt_e4m3", op="norm", rows=16384, n=4096, act="bf16", residual=True,
             quant="block", offset=1.0),
        # a decode step of 96 sequences storing one token each, quantised
        dict(name="append_step_e4m3", op="append", heads=8, dim=128, page=16, kv="e4m3", seqs=96,
             new_lo=1, new_hi=1, old_lo=0, old_hi=2000, lens_seed=4),
        # admitted prompts of ragged lengths stored in an 8-bit cache
        dict(name="append_prompts_e4m3", op="append", heads=2, dim=256, page=64, kv="e4m3", seqs=7,
             new_lo=700, new_hi=9000, old_lo=0, old_hi=100, lens_seed=5),
        # a short cached prefix handed over in bf16
        dict(name="read_short_bf16", op="read", heads=4, dim=64, page=16, kv="bf16", seqs=3,
             new_lo=1, new_hi=300, old_lo=0, old_hi=0, lens_seed=6),
        # whole ragged sequences read back from the 8-bit cache (migration, re-use of a prefix)
        dict(name="read_prefixes_e4m3", op="read", heads=8, dim=128, page=32, kv="e4m3", seqs=11,
             new_lo=500, new_hi=9000, old_lo=0, old_hi=0, lens_seed=7),
        # one sequence's next token over a short history: latency
        dict(name="attn_token", op="attn", q_heads=16, heads=2, dim=256, page=16, kv="bf16", seqs=1,
             new_lo=1, new_hi=1, old_lo=776, old_hi=776, lens_seed=8, gate=True),
        # a decode batch of very uneven histories over the 8-bit cache
        dict(name="attn_decode_ragged_e4m3", op="attn", q_heads=32, heads=8, dim=128, page=16,
             kv="e4m3", seqs=64, new_lo=1, new_hi=1, old_lo=200, old_hi=16000, lens_seed=9,
             gate=False),
        # two long-context sequences decoding: all parallelism is along the cache
        dict(name="attn_decode_long", op="attn", q_heads=16, heads=2, dim=256, page=64, kv="bf16",
             seqs=2, new_lo=1, new_hi=1, old_lo=100003, old_hi=131000, lens_seed=10, gate=True),
        # a mixed batch: chunks of prompts beside decoding rows, 8-bit cache
        dict(name="attn_mixed_e4m3", op="attn", q_heads=16, heads=2, dim=256, page=32, kv="e4m3",
             seqs=12, new_lo=1, new_hi=2500, old_lo=0, old_hi=9000, lens_seed=11, gate=True),
        # a long prompt's chunk after sixteen thousand cached tokens
        dict(name="attn_prompt_chunk", op="attn", q_heads=32, heads=8, dim=128, page=64, kv="bf16",
             seqs=1, new_lo=4096, new_hi=4096, old_lo=16384, old_hi=16384, lens_seed=12,
             gate=False),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], uniform in the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1)))) - 1)))


def _lens(case):
    """(new tokens, cached tokens including the new ones) of every sequence."""
    rng = random.Random(case["lens_seed"])
    new = [_log_int(rng, case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    return new, [n + _log_int(rng, case["old_lo"], case["old_hi"]) for n in new]


def draw(rng):
    op = rng.choice(["norm", "append", "read", "attn", "attn", "attn"])
    if op == "norm":
        n = _log_int(rng, 64, 8192)
        rows = _log_int(rng, 1, min(16384, (1 << 25) // n))
        return dict(op=op, rows=rows, n=n, act=rng.choice(["bf16", "bf16", "f32"]),
                    residual=rng.random() < 0.7, quant=rng.choice(["none", "row", "block"]),
                    offset=rng.choice([0.0, 1.0]))
    dim = rng.choice([64, 128, 256])
    heads = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    kv = rng.choice(["bf16", "e4m3"])
    seed = rng.randrange(1 << 30)
    if op != "attn":
        seqs = _log_int(rng, 1, 128)
        most = max(1, min(9000, (1 << 25) // (dim * heads * seqs)))
        return dict(op=op, heads=heads, dim=dim, page=page, kv=kv, seqs=seqs, new_lo=1, new_hi=most,
                    old_lo=0, old_hi=rng.choice([0, 1000]), lens_seed=seed)
    group = rng.choice([1, 2, 4, 6, 8])
    case = dict(op=op, q_heads=heads * group, heads=heads, dim=dim, page=page, kv=kv, new_lo=1,
                lens_seed=seed, gate=rng.random() < 0.5)
    if rng.random() < 0.5:      # decode: one to a few tokens a sequence over histories of any length
        seqs = _log_int(rng, 1, 64)
        hi = max(64, (1 << 27) // (dim * heads * seqs))
        return dict(case, seqs=seqs, new_hi=rng.choice([1, 1, 4]), old_lo=rng.choice([0, 100]),
                    old_hi=min(hi, 100000))
    seqs = _log_int(rng, 1, 12)  # chunks of prompts
    new = max(1, min(4096, 8192 // seqs) * 4096 // max(4096, dim * case["q_heads"]))
    return dict(case, seqs=seqs, new_hi=new, old_lo=0, old_hi=min(16384, (1 << 15) // seqs))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _quantise(x):
    """x [..., D] in 32 bits -> (e4m3 values, exponent bytes): each vector divided by the least
    power of two 2^(b - 127), 10 <= b, that brings its largest magnitude to 448 or below."""
    amax = x.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(amax)                       # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, torch.zeros_like(e)).clamp(min=-117)
    q = torch.ldexp(x, -e).to(E4M3)
    return q, (e + 127).squeeze(-1).to(torch.uint8)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        act = ACT[case["act"]]
        rows, n = case["rows"], case["n"]
        s["x"] = _randn((rows, n), g, act)
        # a residual stream is larger than what a layer adds, with a few loud channels
        loud = 1.0 + 9.0 * (torch.rand(n, generator=g, device="cuda") < 0.01)
        s["residual"] = (_randn((rows, n), g, torch.float32) * 3.0 * loud).to(act) if case["residual"] else None
        s["weight"] = (_randn((n,), g, torch.float32) * 0.1 + (1.0 - case["offset"])).to(act)
        return s
    new, total = _lens(case)
    H, D, page, n = case["heads"], case["dim"], case["page"], case["seqs"]
    counts = [-(-t // page) for t in total]
    pages = sum(counts) + max(1, sum(counts) // 16)
    order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    table = torch.full((n, max(1, max(counts))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = order[at:at + c]
        at += c
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    s.update(table=table, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
             lens=torch.tensor(total, dtype=torch.int32, device="cuda"), tokens=cu[-1],
             max_new=max(new), max_len=max(total))
    loud = 0.5 + torch.rand((H, 1, 1), generator=g, device="cuda")
    pool = {}
    for name in ("k", "v"):
        x = (torch.randn((pages, H, page, D), generator=g, device="cuda") * loud).to(torch.bfloat16)
        if case["kv"] == "e4m3":
            pool[name + "_pages"], pool[name + "_scales"] = _quantise(x.float())
        else:
            pool[name + "_pages"], pool[name + "_scales"] = x, None
    s.update(pool)
    T = cu[-1]
    if case["op"] == "append":
        # the key and value heads of a fused projection's output: one strided row per token
        kv = _randn((T, 2 * H * D), g)
        s["k"], s["v"] = (kv[:, i * H * D:(i + 1) * H * D].view(T, H, D) for i in range(2))
    if case["op"] == "attn":
        Hq = case["q_heads"]
        if case["gate"]:          # query and output gate of a head side by side, as projected
            qg = _randn((T, Hq, 2 * D), g)
            s["q"], s["gate"] = qg[..., :D], qg[..., D:]
        else:
            s["q"], s["gate"] = _randn((T, Hq, D), g), None
        s["q"].mul_(1.5)
    if own:
        from gated_deltanet_linear_09_gb300 import runtime
        s["cache"] = runtime.PagedKVCache.over(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        s["batch"] = runtime.KVBatch(s["cu"], s["lens"], s["table"], T, s["max_new"])
    return s


# ---------------------------------------------------------------- plain forms (32 bits)

def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    out = []
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out.append(h.to(s["x"].dtype))
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * (s["weight"].float() + c["offset"])
    if c["quant"] == "none":
        return out + [y.to(s["x"].dtype)]
    rows, n = y.shape
    size = n if c["quant"] == "row" else 128
    groups = -(-n // size)
    yp = torch.nn.functional.pad(y, (0, groups * size - n)).view(rows, groups, size)
    scale = (yp.abs().amax(-1) / 448.0).clamp(min=2.0 ** -120)
    q = (yp / scale[..., None]).view(rows, -1)[:, :n].to(E4M3)
    return out + [q, scale]


def _places(s):
    """(page, offset in the page) of every new token, in the order of the packed tokens."""
    t = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["cu"].long(), t, right=True) - 1
    pos = s["lens"].long()[seq] - (s["cu"].long()[seq + 1] - t)
    page = s["case"]["page"]
    return s["table"].long()[seq, pos // page], pos % page


def _plain_append(s):
    at, off = _places(s)
    for name in ("k", "v"):
        pages, scales = s[name + "_pages"], s[name + "_scales"]
        if scales is None:
            pages[at, :, off] = s[name]
        else:
            q, b = _quantise(s[name].float())
            pages.view(torch.uint8)[at, :, off] = q.view(torch.uint8)
            scales[at, :, off] = b
    return [x for x in (s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]) if x is not None]


def _values(pages, scales):
    x = pages.float()
    return x if scales is None else torch.ldexp(x, scales.to(torch.int32)[..., None] - 127)


def _plain_read(s):
    at, off = _places(s)
    out = []
    for name in ("k", "v"):
        pages, scales = s[name + "_pages"], s[name + "_scales"]
        x = pages.view(torch.uint8)[at, :, off].view(E4M3) if scales is not None else pages[at, :, off]
        out.append(_values(x, None if scales is None else scales[at, :, off]).to(torch.bfloat16))
    return out


def _plain_attn(s):
    c = s["case"]
    Hq, H, D, n = c["q_heads"], c["heads"], c["dim"], c["seqs"]
    G, M, L = Hq // H, s["max_new"], s["max_len"]
    table = s["table"].long().clamp(min=0)
    kv = []
    for name in ("k", "v"):      # [n][H][L][D]
        scales = s[name + "_scales"]
        pages = s[name + "_pages"]
        x = pages.view(torch.uint8)[table].view(E4M3) if scales is not None else pages[table]
        x = _values(x, None if scales is None else scales[table])
        kv.append(x.permute(0, 2, 1, 3, 4).reshape(n, H, -1, D)[:, :, :L])
    cu, lens = s["cu"].long(), s["lens"].long()
    t = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    row = t - cu[seq]
    q = torch.zeros((n, M, Hq, D), device="cuda")
    q[seq, row] = s["q"].float()
    q = q.view(n, M, H, G, D).permute(0, 2, 3, 1, 4).reshape(n, H, G * M, D)
    score = (q @ kv[0].transpose(-1, -2)).view(n, H, G, M, L).mul_(1.0 / math.sqrt(D))
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(M, device="cuda")        # [n][M]
    hidden = torch.arange(L, device="cuda")[None, None, :] > pos[:, :, None]           # [n][M][L]
    score.masked_fill_(hidden[:, None, None], -math.inf)
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1, keepdim=True)
    o = (score.view(n, H, G * M, L) @ kv[1]).view(n, H, G, M, D) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(n, M, Hq, D)[seq, row]
    if s["gate"] is not None:
        o = o / (1.0 + torch.exp(-s["gate"].float()))
    return o.to(torch.bfloat16)


def run(s):
    c = s["case"]
    if not own:
        return {"norm": _plain_norm, "append": _plain_append, "read": _plain_read,
                "attn": _plain_attn}[c["op"]](s)
    if c["op"] == "norm":
        from gated_deltanet_linear_09_gb300 import runtime
        y, scales, total = runtime.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=1e-6,
                                            weight_offset=c["offset"], quant=c["quant"])
        return [x for x in (total, y, scales) if x is not None]
    if c["op"] == "append":
        s["cache"].append(s["batch"], s["k"], s["v"])
        return [x for x in (s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]) if x is not None]
    if c["op"] == "read":
        return list(s["cache"].read(s["batch"]))
    return s["cache"].attend(s["batch"], s["q"], gate=s["gate"])


# ---------------------------------------------------------------- work and exact results

def work(case):
    if case["op"] == "norm":
        rows, n = case["rows"], case["n"]
        size = 2 if case["act"] == "bf16" else 4
        b = rows * n * size * (3 if case["residual"] else 1) + n * size
        groups = {"none": 0, "row": 1, "block": -(-n // 128)}[case["quant"]]
        return {"bytes": b + rows * n * (1 if groups else size) + rows * groups * 4, "flops": 6 * rows * n}
    new, total = _lens(case)
    H, D = case["heads"], case["dim"]
    vector = 2 * D if case["kv"] == "bf16" else D + 1
    if case["op"] != "attn":
        return {"bytes": sum(new) * H * 2 * (2 * D + vector), "flops": sum(new) * H * 2 * D}
    Hq = case["q_heads"]
    pairs = sum(a * t - a * (a - 1) // 2 for a, t in zip(new, total))
    return {"bytes": sum(total) * H * 2 * vector + sum(new) * Hq * D * (6 if case["gate"] else 4),
            "flops": 4 * D * Hq * pairs}


def _e4m3_64(x):
    """The nearest e4m3 value of x in 64 bits (ties to even), |x| <= 448."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.sign(x) * torch.round(a / step) * step


def _exact_quant(x):
    amax = x.abs().amax(-1, keepdim=True)
    b = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / 448.0))
    b = torch.where(amax > torch.exp2(b) * 448.0, b + 1, b)
    b = torch.where(amax <= torch.exp2(b - 1) * 448.0, b - 1, b)
    b = torch.where(amax > 0, b, torch.zeros_like(b)).clamp(min=-117.0)
    return _e4m3_64(x / torch.exp2(b))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        out = []
        if s["residual"] is not None:
            h = h + s["residual"].double()
            out.append(h)
        y = h / torch.sqrt((h ** 2).mean(1, keepdim=True) + 1e-6) * (s["weight"].double() + case["offset"])
        if case["quant"] == "none":
            return out + [y]
        n = case["n"]
        size = n if case["quant"] == "row" else 128
        q, scale = [], []
        for c0 in range(0, n, size):
            part = y[:, c0:c0 + size]
            a = part.abs().max(1, keepdim=True).values
            u = torch.clamp(a / 448.0, min=2.0 ** -120)
            scale.append(u)
            q.append(_e4m3_64(part / u))
        return out + [torch.cat(q, 1), torch.cat(scale, 1)]
    new, total = _lens(case)
    page, D, H = case["page"], case["dim"], case["heads"]
    table = s["table"].tolist()

    def place(i, pos):
        return (torch.tensor([table[i][p // page] for p in pos], device="cuda", dtype=torch.int64),
                torch.tensor([p % page for p in pos], device="cuda", dtype=torch.int64))

    def cached(name, i, pos):     # [len(pos)][H][D]
        at, off = place(i, pos)
        scales = s[name + "_scales"]
        if scales is None:
            return s[name + "_pages"][at, :, off].double()
        x = s[name + "_pages"].view(torch.uint8)[at, :, off].view(E4M3).double()
        return x * torch.exp2(scales[at, :, off].double() - 127.0)[..., None]

    at = 0
    if case["op"] == "append":
        pools = {}
        for name in ("k", "v"):
            pools[name] = s[name + "_pages"].double()
            j = 0
            for i, (a, t) in enumerate(zip(new, total)):
                if a:
                    p, o = place(i, list(range(t - a, t)))
                    x = s[name][j:j + a].double()
                    pools[name][p, :, o] = x if case["kv"] == "bf16" else _exact_quant(x)
                j += a
        out = [pools["k"], pools["v"]]
        return out if case["kv"] == "bf16" else out + [None, None]
    if case["op"] == "read":
        return [torch.cat([cached(name, i, list(range(t - a, t))) for i, (a, t) in enumerate(zip(new, total)) if a])
                for name in ("k", "v")]
    Hq = case["q_heads"]
    G = Hq // H
    out = torch.zeros((sum(new), Hq, D), dtype=torch.float64, device="cuda")
    for i, (a, t) in enumerate(zip(new, total)):
        K, V = (cached(name, i, list(range(t))) for name in ("k", "v"))
        for h in range(Hq):
            for r0 in range(0, a, 2048):
                r1 = min(a, r0 + 2048)
                last = t - a + r1        # keys that the last of these rows sees
                sc = s["q"][at + r0:at + r1, h].double() @ K[:last, h // G].T / math.sqrt(D)
                rows = torch.arange(t - a + r0, t - a + r1, device="cuda")
                sc = torch.where(torch.arange(last, device="cuda")[None] <= rows[:, None], sc, -math.inf)
                out[at + r0:at + r1, h] = torch.softmax(sc, -1) @ V[:last, h // G]
        at += a
    if s["gate"] is not None:
        out *= torch.sigmoid(s["gate"].double())
    return out
