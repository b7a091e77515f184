"""Timed cases of the operators between a layer's projections: rotary positions, the paged cache's append
with the heads' norm and rotation on the way, the norms around a block with its gate and residual scale, and
linear attention with a decay for each head (single tokens on the slots' states, and whole prompts).
``own`` selects the library's kernels; otherwise the same results are computed by elementary torch
operations in 32 bits.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decoded token's queries and keys, a quarter of the head rotated: latency
        dict(name="rotary_token", op="rotary", tokens=1, q_heads=16, k_heads=2, dim=256, rot=64, act="bf16",
             interleaved=False, base=1e7, scaling="none", factor=1.0, last=5000),
        # f32 heads of an odd width, adjacent pairs, positions divided by a factor
        dict(name="rotary_odd_f32", op="rotary", tokens=1777, q_heads=5, k_heads=5, dim=81, rot=54, act="f32",
             interleaved=True, base=1e4, scaling="linear", factor=4.0, last=8191),
        # a long-context prompt, whole heads, frequencies stretched by band, positions to a million
        dict(name="rotary_prompt_far", op="rotary", tokens=16384, q_heads=32, k_heads=8, dim=128, rot=128,
             act="bf16", interleaved=False, base=5e5, scaling="bands", factor=16.0, last=1000000),
        # a decoding step of 96 sequences: norm, rotation and 8-bit storage of a token each
        dict(name="append_step_e4m3", op="append", q_heads=32, heads=8, dim=128, page=16, kv="e4m3", rot=128,
             interleaved=False, norm=True, seqs=96, new_lo=1, new_hi=1, old_lo=0, old_hi=2000, lens_seed=4),
        # admitted prompts of ragged lengths, a quarter of the head rotated, the projection's rows in place
        dict(name="append_prompts", op="append", q_heads=16, heads=2, dim=256, page=64, kv="bf16", rot=64,
             interleaved=False, norm=True, seqs=7, new_lo=700, new_hi=9000, old_lo=0, old_hi=100, lens_seed=5),
        # one token between two blocks: latency
        dict(name="block_token", op="block", rows=1, n=5120, group=5120, act="bf16", gate="none", residual=True,
             post=True, pre=True, channel=False, alpha=0.5),
        # a linear layer's heads normed and gated before the output projection
        dict(name="block_heads", op="block", rows=8192, n=4096, group=128, act="bf16", gate="silu",
             residual=False, post=True, pre=False, channel=False, alpha=1.0),
        # a prompt batch between two blocks: norm after, channel scales, residual, norm before the next
        dict(name="block_prompt", op="block", rows=8192, n=5120, group=5120, act="bf16", gate="sigmoid",
             residual=True, post=True, pre=True, channel=True, alpha=1.0),
        # three sequences' next four tokens each (a draft being checked), small heads, decays of the tokens
        dict(name="decay_step_few", op="step", rows=3, tokens=4, k_heads=4, v_heads=8, dk=64, dv=128, slots=5,
             gated=True),
        # a decoding step of 64 sequences
        dict(name="decay_step_batch", op="step", rows=64, tokens=1, k_heads=16, v_heads=48, dk=128, dv=128,
             slots=72, gated=False),
        # one prompt
        dict(name="decay_prompt", op="prompt", k_heads=16, v_heads=32, dk=128, dv=128, seqs=1, lo=4096, hi=4096,
             init=False, gated=False, lens_seed=6),
        # admitted prompts of ragged lengths, some of them continued, decays of the tokens
        dict(name="decay_prompts_ragged", op="prompt", k_heads=16, v_heads=32, dk=128, dv=128, seqs=14, lo=1,
             hi=8192, init=True, gated=True, lens_seed=7),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], uniform in the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1)))) - 1)))


def _lens(case):
    """Cached or state-carried lengths: (new tokens, total tokens) of every sequence."""
    rng = random.Random(case["lens_seed"])
    if case["op"] == "prompt":
        new = [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["seqs"])]
        return new, new
    new = [_log_int(rng, case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    return new, [n + _log_int(rng, case["old_lo"], case["old_hi"]) for n in new]


def draw(rng):
    op = rng.choice(["rotary", "append", "block", "step", "prompt", "prompt"])
    seed = rng.randrange(1 << 30)
    if op == "rotary":
        act = rng.choice(["bf16", "bf16", "f32"])
        dim = rng.choice([64, 80, 128, 256, rng.randrange(16, 257)])
        rot = 2 * rng.choice([dim // 2, dim // 4, max(1, dim // 8)])
        q_heads, k_heads = rng.choice([1, 7, 16, 32]), rng.choice([0, 1, 2, 8])
        most = max(1, min(16384, (1 << 25) // ((q_heads + k_heads) * dim)))
        scaling = rng.choice(["none", "linear", "base", "bands"])
        return dict(op=op, tokens=_log_int(rng, 1, most), q_heads=q_heads, k_heads=k_heads, dim=dim, rot=rot, act=act,
                    interleaved=rng.random() < 0.5, base=rng.choice([1e4, 5e5, 1e7]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0]),
                    last=rng.choice([4096, 131072, 1000000]))
    if op == "append":
        dim, heads = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8])
        q_heads = heads * rng.choice([1, 2, 6, 8])
        kv = rng.choice(["bf16", "bf16", "e4m3"])
        seqs = _log_int(rng, 1, 128)
        most = (1 << 26 if kv == "bf16" else 1 << 22) // (dim * (q_heads + 2 * heads) * seqs)
        return dict(op=op, q_heads=q_heads, heads=heads, dim=dim, page=rng.choice([16, 32, 64, 128]), kv=kv,
                    rot=16 * rng.randrange(1, dim // 16 + 1), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.7, seqs=seqs, new_lo=1, new_hi=max(1, min(9000, most)), old_lo=0,
                    old_hi=rng.choice([0, 1000]), lens_seed=seed)
    if op == "block":
        act = rng.choice(["bf16", "bf16", "f32"])
        post, pre = rng.random() < 0.8, rng.random() < 0.6
        if rng.random() < 0.4:
            group = rng.choice([64, 128, 256])
            n = group * rng.randrange(1, 8192 // group + 1)
        else:
            n = group = _log_int(rng, 64, 8192)
        residual = pre or rng.random() < 0.7
        return dict(op=op, rows=_log_int(rng, 1, min(16384, (1 << 24) // n)), n=n, group=group, act=act,
                    gate=rng.choice(["none", "sigmoid", "silu"]), residual=residual, post=post, pre=pre,
                    channel=rng.random() < 0.3, alpha=rng.choice([1.0, 0.25]))
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64)])
    k_heads = rng.choice([1, 2, 4, 8, 16])
    v_heads = k_heads * rng.choice([1, 2, 3])
    gated = rng.random() < 0.5
    if op == "step":
        rows = _log_int(rng, 1, max(1, min(64, 2048 // v_heads)))
        return dict(op=op, rows=rows, tokens=rng.choice([1, 1, 2, 5, 8]), k_heads=k_heads, v_heads=v_heads, dk=dk, dv=dv,
                    slots=rows + rng.randrange(0, 8), gated=gated)
    seqs = _log_int(rng, 1, 32)
    return dict(op=op, k_heads=k_heads, v_heads=v_heads, dk=dk, dv=dv, seqs=seqs, lo=1,
                hi=max(1, min(16384, (1 << 17) // (v_heads * seqs))), init=rng.random() < 0.5, gated=gated, lens_seed=seed)


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
    return torch.ldexp(x, -e).to(E4M3), (e + 127).squeeze(-1).to(torch.uint8)


def _frequencies(rot, base, scaling, factor, trained=8192):
    """(radians a position of each pair, factor of the rotated values), in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "base":                          # a larger base stretches the slow pairs only
        base = base * factor ** (rot / max(2, rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling != "bands":
        return f, 1.0
    # fast pairs stay, slow ones are stretched, a ramp between: 32 turns and 1 turn in the trained length
    lo, hi = (rot * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (32.0, 1.0))
    lo, hi = max(0.0, math.floor(lo)), min(rot - 1.0, math.ceil(hi))
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
    return f * (1.0 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


def _prepare_rotary(case, g):
    T, D = case["tokens"], case["dim"]
    dt, n = ACT[case["act"]], case["q_heads"] + case["k_heads"]
    qk = _randn((T, n * D), g, dt)                 # the heads of a fused projection's rows
    s = dict(case=case, q=qk[:, :case["q_heads"] * D].view(T, -1, D),
             k=qk[:, case["q_heads"] * D:].view(T, -1, D) if case["k_heads"] else None)
    first = max(0, case["last"] + 1 - T)
    s["pos"] = torch.arange(first, first + T, dtype=torch.int32, device="cuda")
    s["freq"], s["mag"] = _frequencies(case["rot"], case["base"], case["scaling"], case["factor"])
    if own:
        from gated_deltanet_linear_09_gb300 import runtime
        s["plan"] = runtime.Rotary(case["rot"], base=case["base"], interleaved=case["interleaved"],
                                   scaling=case["scaling"], factor=case["factor"], trained=8192)
    else:
        s["freq"] = s["freq"].cuda()
    return s


def _prepare_append(case, g):
    s = dict(case=case)
    new, total = _lens(case)
    H, Hq, D, page, n = case["heads"], case["q_heads"], case["dim"], case["page"], case["seqs"]
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
    T = cu[-1]
    s.update(table=table, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
             lens=torch.tensor(total, dtype=torch.int32, device="cuda"), tokens=T)
    for name in ("k", "v"):
        x = torch.randn((pages, H, page, D), generator=g, device="cuda").to(torch.bfloat16)
        s[name + "_pages"], s[name + "_scales"] = _quantise(x.float()) if case["kv"] == "e4m3" else (x, None)
    # a projection's rows: a head's query beside its gate, then the keys, then the values
    row = _randn((T, (2 * Hq + 2 * H) * D), g)
    s["q"] = row[:, :2 * Hq * D].view(T, Hq, 2 * D)[..., :D]
    s["k"], s["v"] = (row[:, (2 * Hq + i * H) * D:(2 * Hq + (i + 1) * H) * D].view(T, H, D) for i in range(2))
    s["q_norm"], s["k_norm"] = (_randn((D,), g, torch.float32).mul(0.1).to(torch.bfloat16) if case["norm"] else None
                                for _ in range(2))
    s["freq"], s["mag"] = _frequencies(case["rot"], 1e7, "none", 1.0)
    if own:
        from gated_deltanet_linear_09_gb300 import runtime
        s["plan"] = runtime.Rotary(case["rot"], base=1e7, interleaved=case["interleaved"])
        s["cache"] = runtime.PagedKVCache.over(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
        s["batch"] = runtime.KVBatch(s["cu"], s["lens"], s["table"], T, max(new))
    else:
        s["freq"] = s["freq"].cuda()
    return s


def _prepare_block(case, g):
    act, rows, n = ACT[case["act"]], case["rows"], case["n"]
    s = dict(case=case, x=_randn((rows, n), g, act), gate=None, residual=None, post=None, pre=None, channel=None)
    if case["gate"] != "none":
        s["gate"] = _randn((rows, n), g, act)
    if case["residual"]:       # larger than what a block adds, with a few loud channels
        loud = 1.0 + 9.0 * (torch.rand(n, generator=g, device="cuda") < 0.01)
        s["residual"] = (_randn((rows, n), g, torch.float32) * 3.0 * loud).to(act)
    if case["post"]:
        s["post"] = (_randn((case["group"],), g, torch.float32) * 0.1).to(act)
    if case["pre"]:
        s["pre"] = (_randn((n,), g, torch.float32) * 0.1).to(act)
    if case["channel"]:
        s["channel"] = (_randn((n,), g, torch.float32) * 0.05 + 0.2).to(act)
    return s


def _decays(case, shape, g):
    """Log decays: a constant for each head (windows of two to some hundreds of tokens), or of each token by
    a softplus of its own input."""
    H = case["v_heads"]
    if not case["gated"]:
        return -torch.exp2(-8.0 * (torch.arange(H, device="cuda") + 1.0) / H)
    rate = torch.rand((H,), generator=g, device="cuda") * 1.5 + 0.01
    return -rate * torch.nn.functional.softplus(torch.randn((*shape, H), generator=g, device="cuda") - 1.0)


def _prepare_decay(case, g):
    s = dict(case=case)
    Hk, Hv, dk, dv = case["k_heads"], case["v_heads"], case["dk"], case["dv"]
    if case["op"] == "step":
        lead, n = (case["rows"], case["tokens"]), case["rows"]
        slots = case["slots"]
    else:
        new, _ = _lens(case)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        lead, n = (cu[-1],), len(new)
        slots = n + 2
        s.update(cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), lens=new,
                 init=torch.tensor([case["init"] and i % 3 != 1 for i in range(n)], dtype=torch.uint8, device="cuda"))
    s["slots"] = torch.randperm(slots, generator=g, device="cuda")[:n].to(torch.int32)
    row = _randn((*lead, 2 * Hk * dk + Hv * dv), g)          # a projection's rows
    s["q"] = row[..., :Hk * dk].unflatten(-1, (Hk, dk))
    s["k"] = row[..., Hk * dk:2 * Hk * dk].unflatten(-1, (Hk, dk))
    s["v"] = row[..., 2 * Hk * dk:].unflatten(-1, (Hv, dv))
    s["decay"] = _decays(case, lead, g)
    s["state"] = torch.randn((slots, Hv, dk, dv), generator=g, device="cuda")
    if own:
        from gated_deltanet_linear_09_gb300 import runtime
        s["layer"] = runtime.DecayAttention.over(s["state"], Hk)
    return s


def prepare(case, seed):
    g = _gen(seed)
    return {"rotary": _prepare_rotary, "append": _prepare_append, "block": _prepare_block, "step": _prepare_decay,
            "prompt": _prepare_decay}[case["op"]](case, g)


# ---------------------------------------------------------------- plain forms (32 bits)

def _rotate(x, pos, freq, mag, interleaved):
    """x [T][heads][D] in 32 bits; the angles in 64."""
    angle = pos.double()[:, None] * freq[None, :]
    cos, sin = ((f(angle) * mag).float()[:, None] for f in (torch.cos, torch.sin))
    h = freq.shape[0]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y[..., :h], y[..., h:2 * h] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_rotary(s):
    c = s["case"]
    return [_rotate(s[n].float(), s["pos"], s["freq"], s["mag"], c["interleaved"]).to(s[n].dtype)
            for n in ("q", "k") if s[n] is not None]


def _places(s):
    """(page, offset in the page, position) of every new token, in the order of the packed tokens."""
    t = torch.arange(s["tokens"], device="cuda")
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = s["lens"].long()[seq] - (cu[seq + 1] - t)
    page = s["case"]["page"]
    return s["table"].long()[seq, pos // page], pos % page, pos


def _plain_append(s):
    c = s["case"]
    at, off, pos = _places(s)
    out = []
    for name in ("q", "k"):
        x = s[name].float()
        if s[name + "_norm"] is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (s[name + "_norm"].float() + 1.0)
        out.append(_rotate(x, pos, s["freq"], s["mag"], c["interleaved"]))
    for name, x in (("k", out[1]), ("v", s["v"].float())):
        pages, scales = s[name + "_pages"], s[name + "_scales"]
        if scales is None:
            pages[at, :, off] = x.to(torch.bfloat16)
        else:
            q, b = _quantise(x)
            pages.view(torch.uint8)[at, :, off] = q.view(torch.uint8)
            scales[at, :, off] = b
    return [out[0].to(torch.bfloat16)] + [x for x in (s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
                                          if x is not None]


def _plain_block(s):
    c = s["case"]
    x = s["x"].float()
    rows, n = x.shape
    if s["post"] is not None:
        x = x.view(rows, -1, c["group"])
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (s["post"].float() + 1.0)
        x = x.reshape(rows, n)
    if s["gate"] is not None:
        z = s["gate"].float()
        x = x * (1.0 / (1.0 + torch.exp(-z))) * (z if c["gate"] == "silu" else 1.0)
    x = x * c["alpha"]
    if s["channel"] is not None:
        x = x * s["channel"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    out = [x.to(s["x"].dtype)]
    if s["pre"] is not None:
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (s["pre"].float() + 1.0)
        out.append(y.to(s["x"].dtype))
    return out


def _heads(s, name):
    """[..., T][heads][dim] -> 32 bits, a key head repeated for its value heads."""
    x = s[name].float()
    return x if name == "v" else x.repeat_interleave(s["case"]["v_heads"] // s["case"]["k_heads"], -2)


def _plain_step(s):
    c = s["case"]
    q, k, v = (_heads(s, n) for n in ("q", "k", "v"))
    g = s["decay"].expand(*q.shape[:2], c["v_heads"])
    slots = s["slots"].long()
    S = s["state"][slots]
    out = []
    for t in range(c["tokens"]):
        S = S * torch.exp(g[:, t])[..., None, None] + k[:, t, :, :, None] * v[:, t, :, None, :]
        out.append((S * q[:, t, :, :, None]).sum(-2) / math.sqrt(c["dk"]))
    s["state"][slots] = S
    return [torch.stack(out, 1).to(torch.bfloat16), s["state"]]


def _plain_prompt(s):
    """Chunks of 64 tokens of all sequences at once, the sequences padded to the longest."""
    c, C = s["case"], 64
    lens, cu = s["lens"], s["cu"].long()
    n, M, H = len(lens), -(-max(lens) // C) * C, c["v_heads"]
    t = torch.arange(sum(lens), device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    row = t - cu[seq]

    def padded(x):
        y = torch.zeros((n, M, *x.shape[1:]), device="cuda")
        y[seq, row] = x
        return y.transpose(1, 2)                             # [n][H][M](...)
    q, k, v = (padded(_heads(s, name)) for name in ("q", "k", "v"))
    g = padded(s["decay"].expand(sum(lens), H))              # 0 in the padding: the state stays
    slots = s["slots"].long()
    S = s["state"][slots] * s["init"].float()[:, None, None, None]
    later = torch.arange(C, device="cuda")[:, None] < torch.arange(C, device="cuda")[None]
    out = []
    for at in range(0, M, C):
        qc, kc, vc = (x[:, :, at:at + C] for x in (q, k, v))
        gc = torch.cumsum(g[:, :, at:at + C], -1)
        w = torch.exp((gc[..., :, None] - gc[..., None, :]).masked_fill(later, -math.inf))
        o = (qc @ kc.transpose(-1, -2) * w) @ vc + qc @ S * torch.exp(gc)[..., None]
        out.append(o / math.sqrt(c["dk"]))
        rest = torch.exp(gc[..., -1:] - gc)[..., None]
        S = S * torch.exp(gc[..., -1])[..., None, None] + (kc * rest).transpose(-1, -2) @ vc
    s["state"][slots] = S
    return [torch.cat(out, 2).transpose(1, 2)[seq, row].to(torch.bfloat16), s["state"]]


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"rotary": _plain_rotary, "append": _plain_append, "block": _plain_block, "step": _plain_step,
                "prompt": _plain_prompt}[op](s)
    if op == "rotary":
        return [x for x in s["plan"].apply(s["pos"], s["q"], s["k"]) if x is not None]
    if op == "append":
        q = s["cache"].append_rotated(s["batch"], s["plan"], s["q"], s["k"], s["v"], q_norm=s["q_norm"],
                                      k_norm=s["k_norm"], eps=EPS, weight_offset=1.0)
        return [x for x in (q, s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]) if x is not None]
    if op == "block":
        from gated_deltanet_linear_09_gb300 import runtime
        total, y = runtime.block_norm(s["x"], post=s["post"], gate=s["gate"], gate_act=c["gate"], scale=c["alpha"],
                                      channel_scale=s["channel"], residual=s["residual"], pre=s["pre"], eps=EPS,
                                      weight_offset=1.0)
        return [x for x in (total, y) if x is not None]
    if op == "step":
        return [s["layer"].step(s["slots"], s["q"], s["k"], s["v"], s["decay"]), s["state"]]
    return [s["layer"].prefill(s["cu"], s["slots"], s["init"], s["q"], s["k"], s["v"], s["decay"]), s["state"]]


# ---------------------------------------------------------------- work and exact results

def work(case):
    op = case["op"]
    if op == "rotary":
        x = case["tokens"] * (case["q_heads"] + case["k_heads"])
        return {"bytes": 2 * x * case["dim"] * (2 if case["act"] == "bf16" else 4) + 4 * case["tokens"],
                "flops": 3 * x * case["rot"]}
    if op == "append":
        T, H, Hq, D = sum(_lens(case)[0]), case["heads"], case["q_heads"], case["dim"]
        vector = 2 * D if case["kv"] == "bf16" else D + 1
        return {"bytes": T * (Hq * 4 * D + H * (4 * D + 2 * vector)), "flops": T * (Hq + H) * (3 * case["rot"] + 5 * D)}
    if op == "block":
        e = case["rows"] * case["n"]
        planes = 2 + (case["gate"] != "none") + case["residual"] + case["pre"]
        return {"bytes": e * planes * (2 if case["act"] == "bf16" else 4), "flops": 12 * e}
    Hk, Hv, dk, dv = case["k_heads"], case["v_heads"], case["dk"], case["dv"]
    if op == "step":
        tokens, states = case["rows"] * case["tokens"], 2 * case["rows"]
    else:
        lens = _lens(case)[0]
        tokens, states = sum(lens), len(lens) + sum(case["init"] and i % 3 != 1 for i in range(len(lens)))
    io = tokens * (2 * (2 * Hk * dk + 2 * Hv * dv) + (4 * Hv if case["gated"] else 0))
    return {"bytes": io + 4 * states * Hv * dk * dv, "flops": 4 * tokens * Hv * dk * dv}


def _e4m3_64(x):
    """The nearest e4m3 value of x in 64 bits (ties to even), |x| <= 448."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6.0) - 3.0)
    return torch.sign(x) * torch.round(a / step) * step


def _exact_quant(x):
    amax = x.abs().amax(-1, keepdim=True)
    b = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / 448.0))
    b = torch.where(amax > torch.exp2(b) * 448.0, b + 1, b)
    b = torch.where(amax <= torch.exp2(b - 1) * 448.0, b - 1, b)
    b = torch.where(amax > 0, b, torch.zeros_like(b)).clamp(min=-117.0)
    return _e4m3_64(x / torch.exp2(b))


def _turned(x, pos, freq, mag, interleaved):
    """The rotation as a product of complex numbers, in 64 bits."""
    h = freq.shape[0]
    head = x[..., :2 * h].double()
    z = torch.complex(head[..., 0::2], head[..., 1::2]) if interleaved else torch.complex(head[..., :h], head[..., h:])
    turn = torch.outer(pos.double(), freq.to(pos.device))
    z = z * torch.polar(torch.full_like(turn, mag), turn)[:, None]
    head = torch.stack((z.real, z.imag), -1).flatten(-2) if interleaved else torch.cat((z.real, z.imag), -1)
    return torch.cat((head, x[..., 2 * h:].double()), -1)


def _exact_block(s):
    c = s["case"]
    b = s["x"].double()
    if s["post"] is not None:
        parts = b.split(c["group"], 1)
        b = torch.cat([p / torch.sqrt((p ** 2).mean(1, keepdim=True) + EPS) * (1.0 + s["post"].double()) for p in parts], 1)
    if c["gate"] == "sigmoid":
        b = b * torch.sigmoid(s["gate"].double())
    if c["gate"] == "silu":
        b = b * torch.nn.functional.silu(s["gate"].double())
    if s["channel"] is not None:
        b = b * s["channel"].double()
    h = c["alpha"] * b + (0.0 if s["residual"] is None else s["residual"].double())
    if s["pre"] is None:
        return [h]
    return [h, h / torch.sqrt((h ** 2).mean(1, keepdim=True) + EPS) * (1.0 + s["pre"].double())]


def _exact_decay(s):
    """Token by token; the sequences that have run out keep their state."""
    c = s["case"]
    rep = c["v_heads"] // c["k_heads"]
    state = s["state"].double()
    slots = s["slots"].long()
    S = state[slots]
    if c["op"] == "step":
        starts = torch.arange(c["rows"], device="cuda") * c["tokens"]
        lens = torch.full_like(starts, c["tokens"])
    else:
        S = S * s["init"].double()[:, None, None, None]
        starts, lens = s["cu"].long()[:-1], s["cu"].long().diff()
    q, k, v = (s[n].reshape(-1, *s[n].shape[-2:]) for n in ("q", "k", "v"))
    g = s["decay"].expand(*s["q"].shape[:-2], c["v_heads"]).reshape(-1, c["v_heads"])
    out = torch.zeros(v.shape, dtype=torch.float64, device="cuda")
    order = torch.argsort(lens, descending=True)             # the longest first: those still running lead
    S, starts = S[order], starts[order]
    counts = sorted(lens.tolist(), reverse=True)
    for t in range(counts[0]):
        m = sum(x > t for x in counts)
        at = starts[:m] + t
        qt, kt = (x[at].double().repeat_interleave(rep, 1) for x in (q, k))
        live = S[:m]
        live.mul_(torch.exp(g[at].double())[..., None, None]).addcmul_(kt[..., :, None], v[at].double()[..., None, :])
        out[at] = torch.einsum("nhkv,nhk->nhv", live, qt) / math.sqrt(c["dk"])
    state[slots[order]] = S
    return [out.view(*s["v"].shape), state]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "block":
        return _exact_block(s)
    if op in ("step", "prompt"):
        return _exact_decay(s)
    freq, mag, half = s["freq"], s["mag"], case["interleaved"]
    if op == "rotary":
        return [_turned(s[n], s["pos"], freq, mag, half) for n in ("q", "k") if s[n] is not None]
    new, total = _lens(case)
    pos = torch.cat([torch.arange(t - a, t, device="cuda") for a, t in zip(new, total)])
    at = torch.cat([s["table"][i, torch.arange(t - a, t, device="cuda") // case["page"]] for i, (a, t) in
                    enumerate(zip(new, total))]).long()
    vals = {}
    for name in ("q", "k"):
        x = s[name].double()
        if s[name + "_norm"] is not None:
            x = x / torch.sqrt((x ** 2).mean(2, keepdim=True) + EPS) * (1.0 + s[name + "_norm"].double())
        vals[name] = _turned(x, pos, freq, mag, half)
    pools = []
    for name, x in (("k", vals["k"]), ("v", s["v"].double())):
        pool = s[name + "_pages"].double()
        pool[at, :, pos % case["page"]] = x if case["kv"] == "bf16" else _exact_quant(x)
        pools.append(pool)
    return [vals["q"]] + pools + ([] if case["kv"] == "bf16" else [None, None])
