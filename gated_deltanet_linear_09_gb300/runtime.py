"""Device-memory helper around the C ABI: one Gated DeltaNet layer with its slot pool.

Allocation of the weights, the state pool and the prefill workspace happens here (torch owns
device memory); every computation is a call into libgdn.so through ``gdn``.

``stream`` (None: the current one) is where a call runs.  What a call allocates belongs to that
stream, as under ``torch.cuda.stream``; ordering it with others, and ``record_stream`` where another
stream uses a tensor, are the caller's.
"""
from __future__ import annotations

import numpy as np
import torch

from . import gdn
from .synth import BF16, Geometry


def torch_act(geo: Geometry):
    return torch.bfloat16 if geo.act == BF16 else torch.float32


def to_device(x: np.ndarray, dtype, device="cuda") -> torch.Tensor:
    """float32 ndarray holding act-dtype values -> device tensor of that dtype (exact)."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(device=device, dtype=dtype)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """Memory of the stream that is to write it: the allocator gives freed bytes to their stream's next
    tensor, whatever another stream still does with them."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with gdn.on_stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def pack_weight(w: torch.Tensor, stream=None) -> torch.Tensor:
    """A bf16 linear weight [N][K] on the device -> its packed tile layout (uint8 tensor)."""
    nbytes = gdn.gdn_proj_packed_bytes(w.shape[0], w.shape[1])
    if nbytes == 0:
        raise ValueError(f"cannot pack a weight of shape {tuple(w.shape)} (K must be a multiple of 64)")
    packed = _empty((nbytes,), torch.uint8, w.device, stream)
    gdn.gdn_proj_pack(w, packed, stream)
    return packed


class GatedDeltaNetLayer:
    """Weights, state pool (rec f32 [N][Hv][dk][dv], conv act [N][K-1][Cqkv]) and status word."""

    def __init__(self, geo: Geometry, weights: dict, num_slots: int, device="cuda"):
        self.geo = geo
        self.device = device
        self.act = torch_act(geo)
        self.dims = gdn.make_dims(geo.Hk, geo.Hv, geo.dk, geo.dv, geo.K, geo.q_scale, geo.l2_eps,
                                  geo.norm_eps)
        self.A_log = to_device(weights["A_log"], torch.float32, device)
        self.dt_bias = to_device(weights["dt_bias"], torch.float32, device)
        self.conv_w = to_device(weights["conv_w"], self.act, device)
        self.norm_w = to_device(weights["norm_w"], self.act, device)
        self.w = gdn.make_weights(self.A_log, self.dt_bias, self.conv_w, self.norm_w)
        self.rec_state = torch.zeros((num_slots, geo.Hv, geo.dk, geo.dv), dtype=torch.float32,
                                     device=device)
        self.conv_state = torch.zeros((num_slots, geo.K - 1, geo.cqkv), dtype=self.act,
                                      device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.pool = gdn.make_pool(self.rec_state, self.conv_state, self.status)
        self._ws = None
        self.ws_cap = None   # bytes: a smaller prefill workspace (windows of whole chunks)

    @property
    def num_slots(self) -> int:
        return self.rec_state.shape[0]

    def load_state(self, rec: np.ndarray, conv: np.ndarray):
        self.rec_state.copy_(torch.from_numpy(np.ascontiguousarray(rec, np.float32)))
        self.conv_state.copy_(torch.from_numpy(np.ascontiguousarray(conv, np.float32)).to(self.act))

    def inputs(self, xs: dict) -> dict:
        return {k: to_device(v, self.act, self.device) for k, v in xs.items()}

    def decode_step(self, slot_idx: torch.Tensor, qkv, z, a, b, out=None, stream=None):
        if out is None:
            out = _empty((slot_idx.shape[0], self.geo.zdim), self.act, self.device, stream)
        gdn.gdn_decode_step(self.dims, self.w, self.pool, slot_idx, qkv, z, a, b, out, stream)
        return out

    def decode_multi(self, slot_idx: torch.Tensor, qkv, z, a, b, out=None, stream=None):
        """T consecutive tokens per row: qkv [B][T][Cqkv], z [B][T][Hv*dv], a/b [B][T][Hv]."""
        if out is None:
            out = _empty((qkv.shape[0], qkv.shape[1], self.geo.zdim), self.act, self.device, stream)
        gdn.gdn_decode_multi(self.dims, self.w, self.pool, slot_idx, qkv, z, a, b, out, stream)
        return out

    def in_proj(self, hidden: torch.Tensor, w_in_packed: torch.Tensor, stream=None) -> dict:
        """Input projection of bf16 hidden states [rows][H] through the packed stacked weight
        (pack_weight of [Cqkv + Hv*dv + 2*Hv][H]): returns the step inputs qkv, z, a, b."""
        rows, g = hidden.shape[0], self.geo
        dev = hidden.device
        t = {k: _empty((rows, n), torch.bfloat16, dev, stream)
             for k, n in (("qkv", g.cqkv), ("z", g.zdim), ("a", g.Hv), ("b", g.Hv))}
        gdn.gdn_in_proj(self.dims, hidden, w_in_packed, t["qkv"], t["z"], t["b"], t["a"],
                        self.status, stream)
        return t

    def out_proj(self, out: torch.Tensor, w_out_packed: torch.Tensor, hidden_size: int, y=None,
                 stream=None):
        """Output projection of the step's bf16 output [rows][Hv*dv] through the packed
        out_proj weight (pack_weight of [hidden_size][Hv*dv])."""
        if y is None:
            y = _empty((out.shape[0], hidden_size), torch.bfloat16, out.device, stream)
        gdn.gdn_out_proj(self.dims, out, w_out_packed, y, self.status, stream)
        return y

    def conv1d_update(self, slot_idx: torch.Tensor, qkv_in, out=None, stream=None):
        if out is None:
            out = _empty(qkv_in.shape, qkv_in.dtype, qkv_in.device, stream)
        gdn.gdn_conv1d_update(self.dims, self.w, self.pool, slot_idx, qkv_in, out, stream)
        return out

    def workspace(self, num_seqs: int, total_tokens: int, stream=None) -> torch.Tensor:
        need = gdn.gdn_prefill_workspace_bytes(self.dims, num_seqs, total_tokens)
        if self.ws_cap is not None:
            # head dims 128: the prefill runs in windows of whole chunks that fit the workspace
            need = max(gdn.gdn_prefill_workspace_bytes(self.dims, 1, 1), min(need, self.ws_cap))
        if self._ws is None or self._ws.numel() < need:
            self._ws = _empty((max(need, 256),), torch.uint8, self.device, stream)
        return self._ws[:max(need, 256)]

    def prefill(self, cu_seqlens, slot_idx, has_init, qkv, z, a, b, out=None, stream=None):
        """cu_seqlens/slot_idx/has_init: device tensors (int32, int32, uint8 or None)."""
        total = qkv.shape[0]
        n = slot_idx.shape[0]
        if out is None:
            out = _empty((total, self.geo.zdim), self.act, self.device, stream)
        ws = self.workspace(n, total, stream)
        gdn.gdn_prefill_chunked(self.dims, self.w, self.pool, cu_seqlens, slot_idx, has_init, n,
                                total, qkv, z, a, b, out, ws, stream)
        return out

    def compact(self, src, dst, stream=None):
        gdn.gdn_state_compact(self.dims, gdn.act_code(self.act), self.pool, list(src), list(dst),
                              stream)


class _DeviceView:
    """A raw device buffer seen through __cuda_array_interface__ (no copy, no ownership)."""

    def __init__(self, ptr: int, shape, typestr: str):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr,
                                         "data": (int(ptr), False), "version": 2}


class DecodeGraphs:
    """Bucketed CUDA-graph decode over a layer (gdn_decode_graphs_*): write rows [0, B) of the
    static input tensors, call step(B), read rows [0, B) of `out`."""

    def __init__(self, layer: GatedDeltaNetLayer, buckets):
        self.layer = layer
        self.handle = gdn.gdn_decode_graphs_create(layer.dims, layer.w, layer.pool, buckets)
        buf = gdn.gdn_decode_graphs_buffers(self.handle)
        self.max_batch = buf["max_batch"]
        geo, mb = layer.geo, buf["max_batch"]
        ts = "<f2" if layer.act == torch.bfloat16 else "<f4"

        def view(key, shape, typestr, dtype):
            t = torch.as_tensor(_DeviceView(buf[key], shape, typestr), device=layer.device)
            return t.view(dtype) if dtype is not None else t
        act = layer.act if layer.act == torch.bfloat16 else None
        self.slot_idx = view("slot_idx", (mb,), "<i4", None)
        self.qkv = view("qkv", (mb, geo.cqkv), ts, act)
        self.z = view("z", (mb, geo.zdim), ts, act)
        self.a = view("a", (mb, geo.Hv), ts, act)
        self.b = view("b", (mb, geo.Hv), ts, act)
        self.out = view("out", (mb, geo.zdim), ts, act)

    def step(self, B: int, stream=None):
        gdn.gdn_decode_graphs_launch(self.handle, B, stream)
        return self.out[:B]

    def close(self):
        if self.handle:
            torch.cuda.synchronize()
            gdn.gdn_decode_graphs_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------- the full-attention layers' side

_NORM_KINDS = {"none": gdn.GDN_NORM_ACT, "row": gdn.GDN_NORM_E4M3_ROW, "block": gdn.GDN_NORM_E4M3_BLOCK}


def _dense_rows(t) -> bool:
    """The last dimension's elements are adjacent (one element always is)."""
    return t.stride(-1) == 1 or t.shape[-1] <= 1


def rms_norm(x, weight, residual=None, eps=1e-6, weight_offset=0.0, quant="none", stream=None):
    """RMSNorm of x (+ residual), rows [rows][n] of bf16 or f32: returns (y, scales, total).

    total is x + residual in the activation dtype (None without a residual).  quant "none": y in
    the activation dtype, scales None; "row" / "block": y float8_e4m3fn with f32 scales per row
    [rows][1] or per 128 columns [rows][ceil(n / 128)]."""
    shape, dtype = x.shape, x.dtype
    if len(shape) != 2 or not _dense_rows(x) or dtype != weight.dtype or weight.shape != shape[1:] or \
            not _dense_rows(weight):
        raise ValueError("rms_norm takes rows [rows][n] and a weight [n] of one dtype")
    if residual is not None and (residual.shape != shape or residual.dtype != dtype or
                                 not _dense_rows(residual)):
        raise ValueError("residual must have the shape and dtype of x")
    if weight.device != x.device or (residual is not None and residual.device != x.device):
        raise ValueError("x, weight and residual must be on one device")
    kind = _NORM_KINDS.get(quant)
    if kind is None:
        raise ValueError(f"quant is one of {', '.join(_NORM_KINDS)}, not {quant!r}")
    rows, n = shape
    scales = total = None
    if kind == gdn.GDN_NORM_ACT:
        y = _empty(shape, dtype, x.device, stream)
    else:
        y = _empty(shape, torch.float8_e4m3fn, x.device, stream)
        scales = _empty((rows, 1 if quant == "row" else (n + 127) // 128), torch.float32, x.device, stream)
    if residual is not None:
        total = _empty(shape, dtype, x.device, stream)
    gdn.gdn_rms_norm(x, weight, y, residual, total, scales, weight_offset, eps, kind, stream)
    return y, scales, total


class KVBatch:
    """The new tokens of one step: device int32 cu_seqlens [n + 1], kv_lens [n] (cached positions
    including the new tokens) and block_table [n][pages].  total_tokens: packed token rows;
    max_tokens: host bound on one sequence's new tokens (0: unknown)."""

    def __init__(self, cu_seqlens, kv_lens, block_table, total_tokens: int, max_tokens: int = 0):
        for t in (cu_seqlens, kv_lens, block_table):
            if t.dtype != torch.int32 or not _dense_rows(t):
                raise ValueError("cu_seqlens, kv_lens and block_table are int32 with contiguous rows")
        if block_table.dim() != 2 or cu_seqlens.shape[0] != kv_lens.shape[0] + 1 or \
                block_table.shape[0] != kv_lens.shape[0]:
            raise ValueError("cu_seqlens [n + 1], kv_lens [n] and block_table [n][pages] expected")
        if cu_seqlens.dim() != 1 or kv_lens.dim() != 1:
            raise ValueError("cu_seqlens and kv_lens have one dimension")
        self.device = cu_seqlens.device
        if kv_lens.device != self.device or block_table.device != self.device:
            raise ValueError("cu_seqlens, kv_lens and block_table must be on one device")
        self.tensors = (cu_seqlens, kv_lens, block_table)     # kept alive with the struct
        self.total_tokens = int(total_tokens)
        self.c = gdn.make_kv_batch(cu_seqlens, kv_lens, block_table, total_tokens, max_tokens)


class PagedKVCache:
    """Key/value pages [num_pages][num_kv_heads][page_size][head_dim], bf16 or 8-bit e4m3 with one
    power-of-two scale per vector, and the attention workspace of this cache."""

    def __init__(self, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int,
                 quantised: bool = False, device="cuda"):
        shape = (num_pages, num_kv_heads, page_size, head_dim)
        if quantised:
            pages = [torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
                     for _ in range(2)]
            scales = [torch.full(shape[:3], 127, dtype=torch.uint8, device=device) for _ in range(2)]
        else:
            pages = [torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(2)]
            scales = [None, None]
        self._bind(*pages, *scales)

    @classmethod
    def over(cls, k_pages, v_pages, k_scales=None, v_scales=None) -> "PagedKVCache":
        """A cache over existing page tensors."""
        self = cls.__new__(cls)
        self._bind(k_pages, v_pages, k_scales, v_scales)
        return self

    def _bind(self, k_pages, v_pages, k_scales, v_scales):
        q8 = k_pages.dtype == torch.float8_e4m3fn
        if k_pages.dim() != 4 or v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype or \
                not k_pages.is_contiguous() or not v_pages.is_contiguous():
            raise ValueError("k_pages and v_pages: contiguous [pages][heads][page_size][head_dim], one dtype")
        for s in (k_scales, v_scales):
            if (s is not None) != q8 or (q8 and (s.dtype != torch.uint8 or s.shape != k_pages.shape[:3] or
                                                 not s.is_contiguous())):
                raise ValueError("an 8-bit cache has contiguous uint8 scales [pages][heads][page_size]")
        if any(t is not None and t.device != k_pages.device for t in (v_pages, k_scales, v_scales)):
            raise ValueError("pages and scales must be on one device")
        self.k_pages, self.v_pages, self.k_scales, self.v_scales = k_pages, v_pages, k_scales, v_scales
        self.num_kv_heads, self.head_dim = int(k_pages.shape[1]), int(k_pages.shape[3])
        self.device = k_pages.device
        self.status = torch.zeros(1, dtype=torch.int32, device=k_pages.device)
        self.c = gdn.make_kv_cache(k_pages, v_pages, k_scales, v_scales, self.status)
        self._ws, self._ws_need = {}, {}

    def workspace(self, num_q_heads: int, stream=None) -> torch.Tensor:
        """The attention's workspace for this many query heads on this stream.  Calls on one stream
        share it, as long as the cache lives.  A call that is captured in a CUDA graph gets memory of the
        graph's own: graphs captured on one stream may be replayed beside each other."""
        if stream is not None:
            with gdn.on_stream(stream):
                return self._workspace(num_q_heads, gdn.stream_handle())
        return self._workspace(num_q_heads, gdn.stream_handle())

    def _workspace(self, num_q_heads, current):
        need = self._ws_need.get(num_q_heads)
        if need is None:
            need = gdn.gdn_paged_attention_workspace_bytes(self.c, num_q_heads)
            if need == 0:
                raise ValueError(f"{num_q_heads} query heads over this cache are not supported")
            self._ws_need[num_q_heads] = need
        if torch.cuda.is_current_stream_capturing():
            return torch.empty(need, dtype=torch.uint8, device=self.device)
        ws = self._ws.get(current)
        if ws is None or ws.numel() < need:
            ws = self._ws[current] = torch.empty(need, dtype=torch.uint8, device=self.device)
        return ws

    def _check(self, t, batch, what):
        shape, stride = t.shape, t.stride()
        if len(shape) != 3 or shape[0] != batch.total_tokens or shape[2] != self.head_dim or \
                t.dtype != torch.bfloat16 or stride[2] != 1:
            raise ValueError(f"{what}: bf16 [total_tokens][heads][head_dim] with contiguous vectors expected")
        device = self.device
        if t.device != device or batch.device != device:
            raise ValueError(f"{what} is on {t.device}, the batch on {batch.device}, the cache on {device}")
        return shape, stride

    def append(self, batch: KVBatch, k, v, stream=None):
        """Stores the new tokens' keys and values, bf16 [total_tokens][num_kv_heads][head_dim]."""
        for t, what in ((k, "k"), (v, "v")):
            shape, stride = self._check(t, batch, what)
            if shape[1] != self.num_kv_heads or (stride[1] != self.head_dim and self.num_kv_heads > 1):
                raise ValueError(f"{what}: {self.num_kv_heads} adjacent heads expected")
        if batch.total_tokens:
            gdn.gdn_kv_append(self.c, batch.c, k, v, stream)

    def read(self, batch: KVBatch, k=None, v=None, stream=None):
        """The batch's tokens' keys and values back as bf16 (k, v)."""
        shape = (batch.total_tokens, self.num_kv_heads, self.head_dim)
        if k is None:
            k = _empty(shape, torch.bfloat16, self.device, stream)
        elif k.shape != shape or k.dtype != torch.bfloat16 or not k.is_contiguous():
            raise ValueError("k: contiguous bf16 [total_tokens][num_kv_heads][head_dim]")
        if v is None:
            v = _empty(shape, torch.bfloat16, self.device, stream)
        elif v.shape != shape or v.dtype != torch.bfloat16 or not v.is_contiguous():
            raise ValueError("v: contiguous bf16 [total_tokens][num_kv_heads][head_dim]")
        if k.device != self.device or v.device != self.device or batch.device != self.device:
            raise ValueError("the batch, k and v must be on the cache's device")
        if batch.total_tokens:
            gdn.gdn_kv_read(self.c, batch.c, k, v, stream)
        return k, v

    def attend(self, batch: KVBatch, q, gate=None, scale=0.0, out=None, workspace=None, stream=None):
        """Causal attention of the new tokens' queries, bf16 [total_tokens][num_q_heads][head_dim]
        (times sigmoid(gate)), over the cache, which already holds their keys and values."""
        shape, _ = self._check(q, batch, "q")
        if gate is not None and self._check(gate, batch, "gate")[0] != shape:
            raise ValueError("gate must have the shape of q")
        if out is None:
            out = _empty(shape, torch.bfloat16, self.device, stream)
        elif out.shape != shape or out.dtype != torch.bfloat16 or not out.is_contiguous() or out.device != self.device:
            raise ValueError("out: contiguous bf16 with the shape of q, on the cache's device")
        if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous() or
                                      workspace.device != self.device):
            raise ValueError("workspace: contiguous uint8 on the cache's device")
        if batch.total_tokens:
            if workspace is not None:
                pass
            elif stream is None:
                stream = gdn.stream_handle()
                workspace = self._workspace(shape[1], stream)
            else:
                workspace = self.workspace(shape[1], stream)
            gdn.gdn_paged_attention(self.c, batch.c, q, out, workspace, gate, scale, stream)
        return out
