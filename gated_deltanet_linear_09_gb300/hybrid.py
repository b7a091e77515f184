"""One period of a hybrid model's layers, run through the library: Gated DeltaNet layers and one
full-attention layer over a paged cache, each entered through the residual's RMSNorm.

``python -m gated_deltanet_linear_09_gb300.hybrid`` admits a few prompts in pieces, decodes from
them with the decoding step captured in a CUDA graph, and prints the rates.  Linear-attention layers
with a decay for each head (`DecayLayer`) may stand among the Gated DeltaNet ones, and a norm and a scale
after every layer.  The MLPs are the caller's.
"""
from __future__ import annotations

import argparse
import time

import torch

from . import gdn, synth
from .runtime import (DecayAttention, GatedDeltaNetLayer, KVBatch, PagedKVCache, Rotary, block_norm, pack_weight,
                      rms_norm, to_device)


def _linear(x, packed, widths, status):
    """The packed projection of x, its output features in dense tensors of these widths."""
    outs = [torch.empty((x.shape[0], n), dtype=torch.bfloat16, device=x.device) for n in widths]
    route = gdn.make_route([(sum(widths[:i]), n, t) for i, (n, t) in enumerate(zip(widths, outs))])
    gdn.gdn_linear_bf16(x, packed, sum(widths), route, 0, status)
    return outs


class AttentionLayer:
    """Gated full attention: projections, per-head RMSNorm of queries and keys, the cache's append
    and the attention of the new tokens over it.  Weights are bf16 rows as stored: w_q [Hq * 2 * D]
    (a head's query rows, then its gate's), w_k and w_v [Hkv * D], all [..][hidden]; w_out
    [hidden][Hq * D]; q_norm and k_norm [D], counted from 1.  With `rotary` queries and keys are turned to
    their places in the cache, in one launch with the norms and the append."""

    rotary = None

    def __init__(self, cache: PagedKVCache, num_q_heads: int, weights: dict, eps: float = 1e-6, rotary: Rotary = None):
        self.cache, self.Hq, self.eps = cache, num_q_heads, eps
        self.H, self.D = cache.num_kv_heads, cache.head_dim
        self.hidden = weights["w_out"].shape[0]
        self.w_in = pack_weight(torch.cat([weights[k] for k in ("w_q", "w_k", "w_v")]))
        self.w_out = pack_weight(weights["w_out"])
        self.q_norm, self.k_norm = weights["q_norm"], weights["k_norm"]
        self.rotary = rotary
        self.status = torch.zeros(1, dtype=torch.int32, device=cache.device)

    def _linear(self, x, packed, widths):
        return _linear(x, packed, widths, self.status)

    def forward(self, batch: KVBatch, x, rotate=None, stream=None):
        """x: normed hidden states bf16 [total_tokens][hidden].  rotate(q, k) -> (q, k) applies a position
        embedding of the caller's to [tokens][heads][D] tensors, on the stream of the call."""
        if rotate is not None and self.rotary is not None:
            raise ValueError("the layer turns queries and keys itself")
        with gdn.on_stream(stream):
            return self._forward(batch, x, rotate)

    def _forward(self, batch, x, rotate):
        T, Hq, H, D = x.shape[0], self.Hq, self.H, self.D
        qg, k, v = self._linear(x, self.w_in, [Hq * 2 * D, H * D, H * D])
        if self.rotary is not None:
            qg = qg.view(T, Hq, 2 * D)
            q = self.cache.append_rotated(batch, self.rotary, qg[..., :D], k.view(T, H, D), v.view(T, H, D), q_norm=self.q_norm,
                                          k_norm=self.k_norm, eps=self.eps, weight_offset=1.0)
            o = self.cache.attend(batch, q, gate=qg[..., D:])
            return self._linear(o.view(T, Hq * D), self.w_out, [self.hidden])[0]
        qg = qg.view(T * Hq, 2 * D)
        q, _, _ = rms_norm(qg[:, :D], self.q_norm, eps=self.eps, weight_offset=1.0)
        k, _, _ = rms_norm(k.view(T * H, D), self.k_norm, eps=self.eps, weight_offset=1.0)
        q, k = q.view(T, Hq, D), k.view(T, H, D)
        if rotate is not None:
            q, k = rotate(q, k)
        self.cache.append(batch, k, v.view(T, H, D))
        o = self.cache.attend(batch, q, gate=qg.view(T, Hq, 2 * D)[..., D:])
        return self._linear(o.view(T, Hq * D), self.w_out, [self.hidden])[0]


class DecayLayer:
    """Linear attention with a decay for each head: projections, rotary positions (with `rotary`), the attention
    on the slots' states, a norm of each head gated by SiLU, and the output projection.  Weights are bf16 rows
    as stored: w_q and w_k [Hk * dk], w_v and w_z [Hv * dv], all [..][hidden]; w_out [hidden][Hv * dv]; norm
    [dv], counted from 1; log_decay f32 [Hv]."""

    def __init__(self, attention: DecayAttention, weights: dict, eps: float = 1e-6, rotary: Rotary = None):
        self.attention, self.eps, self.rotary = attention, eps, rotary
        self.hidden = weights["w_out"].shape[0]
        self.w_in = pack_weight(torch.cat([weights[k] for k in ("w_q", "w_k", "w_v", "w_z")]))
        self.w_out = pack_weight(weights["w_out"])
        self.norm, self.log_decay = weights["norm"], weights["log_decay"]
        self.status = torch.zeros(1, dtype=torch.int32, device=attention.device)

    def forward(self, x, slots, cu_seqlens=None, has_init=None, positions=None, stream=None):
        """x: normed hidden states bf16 [tokens][hidden], one token per slot without cu_seqlens, else pieces of
        prompts; positions (device int32 [tokens]) with a rotation."""
        if self.rotary is not None and positions is None:
            raise ValueError("a layer with a rotation needs the tokens' positions")
        with gdn.on_stream(stream):
            a = self.attention
            T, qk, vz = x.shape[0], a.Hk * a.dk, a.Hv * a.dv
            q, k, v, z = _linear(x, self.w_in, [qk, qk, vz, vz], self.status)
            q, k, v = q.view(T, a.Hk, a.dk), k.view(T, a.Hk, a.dk), v.view(T, a.Hv, a.dv)
            if self.rotary is not None:
                self.rotary.apply(positions, q, k, q_out=q, k_out=k)
            if cu_seqlens is None:
                o = a.step(slots, q, k, v, self.log_decay)
            else:
                o = a.prefill(cu_seqlens, slots, has_init, q, k, v, self.log_decay)
            y, _ = block_norm(o.view(T, vz), post=self.norm, gate=z, gate_act="silu", eps=self.eps, weight_offset=1.0)
            return _linear(y, self.w_out, [self.hidden], self.status)[0]


class HybridPeriod:
    """Gated DeltaNet layers, or DecayLayers, followed by one AttentionLayer, with the norms between them.
    post_norms: a norm of each linear layer's output (bf16 [hidden], counted from 1), before it is added to the
    residual times residual_scale."""

    post_norms, residual_scale = None, 1.0

    def __init__(self, linear_layers, attention: AttentionLayer, norms, post_norms=None, residual_scale: float = 1.0):
        self.linear_layers = linear_layers          # (GatedDeltaNetLayer, packed in, packed out), or DecayLayer
        self.attention, self.norms = attention, norms
        self.post_norms, self.residual_scale = post_norms, residual_scale

    def step(self, batch: KVBatch, x, slots, cu_seqlens=None, has_init=None, rotate=None, positions=None):
        """x bf16 [tokens][hidden] -> (x, residual): the layers' output and the sum it is to be added
        to.  One token per sequence without cu_seqlens, else pieces of prompts.  positions: device int32
        [tokens], for DecayLayers with a rotation."""
        residual = None
        for i, layer in enumerate(self.linear_layers):
            x, residual = self._enter(x, residual, i)
            if isinstance(layer, DecayLayer):
                x = layer.forward(x, slots, cu_seqlens, has_init, positions)
                continue
            layer, w_in, w_out = layer
            t = layer.in_proj(x, w_in)
            if cu_seqlens is None:
                o = layer.decode_step(slots, t["qkv"], t["z"], t["a"], t["b"])
            else:
                o = layer.prefill(cu_seqlens, slots, has_init, t["qkv"], t["z"], t["a"], t["b"])
            x = layer.out_proj(o, w_out, x.shape[1])
        x, residual = self._enter(x, residual, len(self.linear_layers))
        return self.attention.forward(batch, x, rotate), residual

    def _enter(self, x, residual, i):
        """The norm before layer i, of the sum of what came before it."""
        if residual is not None and (self.post_norms is not None or self.residual_scale != 1.0):
            total, y = block_norm(x, post=self.post_norms[i - 1] if self.post_norms is not None else None, residual=residual,
                                  pre=self.norms[i], scale=self.residual_scale, weight_offset=1.0)
            return y, total
        y, _, total = rms_norm(x, self.norms[i], residual=residual, weight_offset=1.0)
        return y, x if total is None else total


def attention_weights(hidden, num_q_heads, num_kv_heads, head_dim, seed, device="cuda"):
    """Random weights of an AttentionLayer."""
    g = torch.Generator().manual_seed(seed)

    def rows(n, k):
        return (torch.randn((n, k), generator=g) / k ** 0.5).to(device=device, dtype=torch.bfloat16)
    w = {"w_q": rows(num_q_heads * 2 * head_dim, hidden), "w_k": rows(num_kv_heads * head_dim, hidden),
         "w_v": rows(num_kv_heads * head_dim, hidden), "w_out": rows(hidden, num_q_heads * head_dim)}
    for k in ("q_norm", "k_norm"):
        w[k] = (0.1 * torch.randn(head_dim, generator=g)).to(device=device, dtype=torch.bfloat16)
    return w


def decay_weights(hidden, num_k_heads, num_v_heads, head_k_dim, head_v_dim, seed, device="cuda"):
    """Random weights of a DecayLayer; windows of some tokens to some hundreds."""
    g = torch.Generator().manual_seed(seed)
    qk, vz = num_k_heads * head_k_dim, num_v_heads * head_v_dim
    w = {k: (torch.randn((n, m), generator=g) / m ** 0.5).to(device=device, dtype=torch.bfloat16)
         for k, n, m in (("w_q", qk, hidden), ("w_k", qk, hidden), ("w_v", vz, hidden), ("w_z", vz, hidden), ("w_out", hidden, vz))}
    w["norm"] = (0.1 * torch.randn(head_v_dim, generator=g)).to(device=device, dtype=torch.bfloat16)
    w["log_decay"] = -torch.exp2(-8.0 * torch.arange(1, num_v_heads + 1, device=device) / num_v_heads)
    return w


def make_period(geo: synth.Geometry, hidden, cache: PagedKVCache, num_q_heads, num_slots, linear=3, seed=0, decayed=0,
                rotary: Rotary = None, post_norms: bool = False, residual_scale: float = 1.0):
    """A HybridPeriod with random weights; the last `decayed` of its linear layers are DecayLayers of the same
    geometry.  rotary: of the attention layer; DecayLayers then turn whole heads."""
    device = cache.device
    layers = []
    for i in range(linear):
        if i >= linear - decayed:
            attention = DecayAttention(geo.Hk, geo.Hv, geo.dk, geo.dv, num_slots, device=device)
            weights = decay_weights(hidden, geo.Hk, geo.Hv, geo.dk, geo.dv, seed + i, device)
            layers.append(DecayLayer(attention, weights, rotary=None if rotary is None else Rotary(geo.dk, device=device)))
            continue
        layer = GatedDeltaNetLayer(geo, synth.make_weights(geo, seed + i), num_slots, device)
        w = synth.make_proj_weights(geo, hidden, seed + i)
        layers.append((layer, pack_weight(to_device(w["w_in"], torch.bfloat16, device)),
                       pack_weight(to_device(w["w_out"], torch.bfloat16, device))))
    g = torch.Generator().manual_seed(seed)
    norms = [(0.1 * torch.randn(hidden, generator=g)).to(device=device, dtype=torch.bfloat16)
             for _ in range(linear + 1)]
    weights = attention_weights(hidden, num_q_heads, cache.num_kv_heads, cache.head_dim, seed, device)
    posts = [(0.1 * torch.randn(hidden, generator=g)).to(device=device, dtype=torch.bfloat16)
             for _ in range(linear)] if post_norms else None
    return HybridPeriod(layers, AttentionLayer(cache, num_q_heads, weights, rotary=rotary), norms, posts, residual_scale)


def main(argv=None):
    p = argparse.ArgumentParser(description="a hybrid model's layers over a paged cache")
    p.add_argument("--sequences", type=int, default=16)
    p.add_argument("--prompt", type=int, default=1500, help="tokens of the longest prompt")
    p.add_argument("--piece", type=int, default=1024, help="prompt tokens admitted at once")
    p.add_argument("--steps", type=int, default=32, help="decoding steps")
    p.add_argument("--bf16-cache", action="store_true", help="keep the cache in bf16 instead of 8 bits")
    p.add_argument("--rotary", action="store_true", help="rotary positions on a quarter of the attention layer's heads")
    p.add_argument("--decayed", type=int, default=0, help="linear layers with a decay for each head, of the three")
    p.add_argument("--post-norms", action="store_true", help="a norm after every linear layer")
    a = p.parse_args(argv)
    n, page, hidden = a.sequences, 32, 2048
    geo = synth.Geometry(16, 32, 128, 128)
    prompts = [max(1, a.prompt - 37 * i) for i in range(n)]
    width = -(-(max(prompts) + a.steps + 1) // page)
    cache = PagedKVCache(n * width, page, 2, 256, not a.bf16_cache)
    period = make_period(geo, hidden, cache, 16, n, decayed=min(3, a.decayed), rotary=Rotary(64, base=1e7) if a.rotary else None,
                         post_norms=a.post_norms)
    table = torch.randperm(n * width, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    table = table.view(n, width).cuda()
    g = torch.Generator(device="cuda").manual_seed(2)

    def tokens(count):
        return torch.randn((count, hidden), generator=g, device="cuda").to(torch.bfloat16)

    def ints(xs):
        return torch.tensor(xs, dtype=torch.int32, device="cuda")

    torch.cuda.synchronize()
    start, done = time.perf_counter(), [0] * n
    while any(d < t for d, t in zip(done, prompts)):
        live = [i for i in range(n) if done[i] < prompts[i]]
        new = [min(a.piece, prompts[i] - done[i]) for i in live]
        cu = [sum(new[:i]) for i in range(len(new) + 1)]
        batch = KVBatch(ints(cu), ints([done[i] + m for i, m in zip(live, new)]), table[live], cu[-1], max(new))
        has_init = torch.tensor([done[i] > 0 for i in live], dtype=torch.uint8, device="cuda")
        places = ints([done[i] + j for i, m in zip(live, new) for j in range(m)])
        x, _ = period.step(batch, tokens(cu[-1]), ints(live), ints(cu), has_init, positions=places)
        for i, m in zip(live, new):
            done[i] += m
    torch.cuda.synchronize()
    print(f"prompts: {sum(prompts)} tokens in {1e3 * (time.perf_counter() - start):.1f} ms (first calls included)")

    lens = ints(prompts)
    batch, slots, x = KVBatch(ints(list(range(n + 1))), lens, table, n, 1), ints(list(range(n))), tokens(n)
    places = torch.empty_like(lens)

    def step():
        places.copy_(lens)
        lens.add_(1)
        return period.step(batch, x, slots, positions=places)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    ms = 1e3 * (time.perf_counter() - start) / max(1, a.steps)
    bad = [int(t.status.item()) for t in (cache, period.attention, *(x.attention if isinstance(x, DecayLayer) else x[0]
                                                                       for x in period.linear_layers))]
    print(f"decode: {n} sequences, {ms * 1e3:.1f} us a step, status {bad}, finite {bool(out.isfinite().all())}")
    return 0 if not any(bad) and bool(out.isfinite().all()) else 1


if __name__ == "__main__":
    raise SystemExit(main())
