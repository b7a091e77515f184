"""Device-memory helper around the C ABI: one Gated DeltaNet layer with its slot pool.

Allocation of the weights, the state pool and the prefill workspace happens here (torch owns
device memory); every computation is a call into libgdn.so through ``gdn``.

``stream`` (None: the current one) is where a call runs.  What a call allocates belongs to that
stream, as under ``torch.cuda.stream``; ordering it with others, and ``record_stream`` where another
stream uses a tensor, are the caller's.
"""
from __future__ import annotations

import math

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


class Rotary:
    """Rotary positions: the first rot_dim elements of a head turned in pairs, adjacent ones (interleaved) or
    i and i + rot_dim / 2, pair i by position * base^(-2i / rot_dim) radians.  For contexts `factor` times the
    trained length, scaling "linear" divides every frequency by it; "base" multiplies the base by
    factor^(rot_dim / (rot_dim - 2)), which stretches the slow pairs only; "bands" keeps pairs that make more
    than 32 turns within `trained` positions, divides those that make less than one, ramps between, and
    multiplies what is turned by 0.1 ln(factor) + 1 (by 1 for a factor below 1).  The frequencies are held to
    2^-64 of a turn, so that the angle of any position is exact."""

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, trained: int = 8192, device="cuda"):
        if rot_dim < 2 or rot_dim % 2:
            raise ValueError("rot_dim is even and at least 2")
        if not (base > 1.0 and factor > 0.0 and math.isfinite(base) and math.isfinite(factor)):
            raise ValueError("base > 1 and factor > 0 expected")
        if scaling == "base":
            base = base * factor ** (rot_dim / max(2, rot_dim - 2))
        f = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
        scale = 1.0
        if scaling == "linear":
            f = [x / factor for x in f]
        elif scaling == "bands":
            lo, hi = (rot_dim * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (32.0, 1.0))
            lo, hi = max(0.0, math.floor(lo)), min(rot_dim - 1.0, math.ceil(hi))
            ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(rot_dim // 2)]
            f = [x * (1.0 - r) + x / factor * r for x, r in zip(f, ramp)]
            scale = 0.1 * math.log(max(factor, 1.0)) + 1.0
        elif scaling not in ("none", "base"):
            raise ValueError(f"scaling is none, linear, base or bands, not {scaling!r}")
        self._bind(f, interleaved, scale, device)

    @classmethod
    def of(cls, frequencies, interleaved: bool = False, scale: float = 1.0, device="cuda") -> "Rotary":
        """From each pair's radians a position."""
        self = cls.__new__(cls)
        self._bind([float(x) for x in frequencies], interleaved, float(scale), device)
        return self

    def _bind(self, frequencies, interleaved, scale, device):
        if not frequencies or not all(math.isfinite(x) for x in frequencies) or not math.isfinite(scale):
            raise ValueError("finite frequencies and scale expected")
        self.frequencies, self.rot_dim, self.scale = frequencies, 2 * len(frequencies), scale
        turns = [round(x / (2 * math.pi) * 2.0 ** 64) & (2 ** 64 - 1) for x in frequencies]
        self.turns = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device)
        self.device = self.turns.device
        self.c = gdn.make_rotary(self.turns, self.rot_dim, interleaved, scale)

    def _refuse(self, t, out, tokens, what):
        """Why t, or its output, is not taken."""
        if len(t.shape) != 3 or t.shape[0] != tokens or t.shape[2] < self.rot_dim or not _dense_rows(t):
            raise ValueError(f"{what}: [tokens][heads][dim >= {self.rot_dim}] with contiguous vectors expected")
        if t.device != self.device:
            raise ValueError(f"{what} is on {t.device}, the rotation on {self.device}")
        raise ValueError(f"{what}'s output: contiguous, with its shape and type, on its device")

    def _output(self, t, out, tokens, what, stream):
        """t checked, and its output, a new one or `out`."""
        shape, device = t.shape, self.device
        if len(shape) != 3 or shape[0] != tokens or shape[2] < self.rot_dim or t.stride()[2] != 1 or t.device != device:
            self._refuse(t, out, tokens, what)
        if out is None:
            return _empty(shape, t.dtype, device, stream)
        if out.shape != shape or out.dtype != t.dtype or not out.is_contiguous() or out.device != device:
            self._refuse(t, out, tokens, what)
        return out

    def apply(self, positions, q=None, k=None, q_out=None, k_out=None, stream=None):
        """(q, k) turned at positions (device int32 [tokens]); q and k bf16 or f32 [tokens][heads][dim], either may
        be None.  Outputs may be the inputs where those are contiguous."""
        if positions.dtype != torch.int32 or positions.dim() != 1 or not _dense_rows(positions) or \
                positions.device != self.device:
            raise ValueError("positions: contiguous int32 [tokens] on the rotation's device")
        if (q is None and q_out is not None) or (k is None and k_out is not None):
            raise ValueError("an output without its input")
        tokens = positions.shape[0]
        if q is not None:
            if k is not None and (q.dtype != k.dtype or q.shape[-1] != k.shape[-1]):
                raise ValueError("q and k have one type and head size")
            q_out = self._output(q, q_out, tokens, "q", stream)
        if k is not None:
            k_out = self._output(k, k_out, tokens, "k", stream)
        if q is not None or k is not None:
            gdn.gdn_rotary_apply(self.c, positions, q, q_out, k, k_out, stream)
        return q_out, k_out


_GATES = {"sigmoid": gdn.GDN_GATE_SIGMOID, "silu": gdn.GDN_GATE_SILU}


def block_norm(x, post=None, gate=None, gate_act="sigmoid", scale=1.0, channel_scale=None, residual=None, pre=None,
               eps=1e-6, weight_offset=0.0, total=None, y=None, stream=None):
    """A block's output x [rows][n] (bf16 or f32) on its way to the next block: returns (total, y),
      total = residual + scale * channel_scale * norm(x; post) * act(gate),  y = norm(total; pre),
    whatever of it is given (y None without pre).  post [n] norms the row, a shorter post (32, 64, 128 or 256
    weights) each run of that many columns.  gate_act "sigmoid", or "silu": gate * sigmoid(gate)."""
    shape, dtype, device = x.shape, x.dtype, x.device
    if len(shape) != 2 or not _dense_rows(x):
        raise ValueError("block_norm takes rows [rows][n]")

    def rows(t, what):
        if t.shape != shape or t.dtype != dtype or not _dense_rows(t) or t.device != device:
            raise ValueError(f"{what} must have the shape, type and device of x")
        return t

    def vector(t, what):
        if t.dim() != 1 or t.dtype != dtype or t.device != device or not _dense_rows(t) or \
                (what != "post" and t.shape[0] != shape[1]):
            raise ValueError(f"{what}: a vector of x's type and width on its device")
        return t
    act = gdn.GDN_GATE_NONE
    if gate is not None:
        rows(gate, "gate")
        act = _GATES.get(gate_act)
        if act is None:
            raise ValueError(f"gate_act is sigmoid or silu, not {gate_act!r}")
    if residual is not None:
        rows(residual, "residual")
    group = shape[1] if post is None else vector(post, "post").shape[0]
    if channel_scale is not None:
        vector(channel_scale, "channel_scale")
    if total is None:
        total = _empty(shape, dtype, device, stream)
    elif not rows(total, "total").is_contiguous():
        raise ValueError("total must be contiguous")
    if pre is None:
        if y is not None:
            raise ValueError("y is written with pre only")
    else:
        vector(pre, "pre")
        if y is None:
            y = _empty(shape, dtype, device, stream)
        elif not rows(y, "y").is_contiguous():
            raise ValueError("y must be contiguous")
    gdn.gdn_block_norm(x, total, y, post, gate, act, residual, pre, channel_scale, scale, weight_offset, eps, group, stream)
    return total, y


class DecayAttention:
    """Linear attention with a decay for each head, S = exp(g) S + k v^T, o = scale S^T q, on a pool of states
    f32 [num_slots][num_v_heads][dk][dv]; value head h reads query and key head h * num_k_heads // num_v_heads.
    scale 0: 1/sqrt(dk)."""

    def __init__(self, num_k_heads: int, num_v_heads: int, head_k_dim: int, head_v_dim: int, num_slots: int,
                 scale: float = 0.0, device="cuda"):
        self._bind(torch.zeros((num_slots, num_v_heads, head_k_dim, head_v_dim), dtype=torch.float32, device=device),
                   num_k_heads, scale)

    @classmethod
    def over(cls, state, num_k_heads: int, scale: float = 0.0) -> "DecayAttention":
        """On an existing pool of states."""
        self = cls.__new__(cls)
        self._bind(state, num_k_heads, scale)
        return self

    def _bind(self, state, num_k_heads, scale):
        if state.dim() != 4 or state.dtype != torch.float32 or not state.is_contiguous():
            raise ValueError("state: contiguous f32 [num_slots][num_v_heads][dk][dv]")
        if num_k_heads < 1 or state.shape[1] % num_k_heads:
            raise ValueError("num_v_heads is a multiple of num_k_heads")
        self.state, self.device = state, state.device
        self.Hk, self.Hv, self.dk, self.dv = num_k_heads, *(int(x) for x in state.shape[1:])
        self.status = torch.zeros(1, dtype=torch.int32, device=state.device)
        self.c = gdn.make_decay_layer(state, num_k_heads, scale, self.status)
        self._ws = {}

    @staticmethod
    def _distance(strides, lead, dense, what):
        """The distance of the tokens that the leading dimensions count (1, or rows and their T tokens); that of a
        dimension of size one says nothing."""
        if len(lead) == 1:
            return strides[0] if lead[0] > 1 else dense
        rows, T = lead
        if T == 1:
            return strides[0] if rows > 1 else dense
        if rows > 1 and strides[0] != T * strides[1]:
            raise ValueError(f"{what}: its tokens must lie at one distance from each other")
        return strides[1]

    def _tokens(self, lead, q, k, v, log_decay, out, stream):
        """(tokens struct, out) of tensors [*lead][heads][dim], without a copy."""
        device, distances = self.device, []
        for t, what, heads, dim in ((q, "q", self.Hk, self.dk), (k, "k", self.Hk, self.dk), (v, "v", self.Hv, self.dv)):
            if t.shape != (*lead, heads, dim) or t.dtype != torch.bfloat16 or t.device != device:
                raise ValueError(f"{what}: bf16 {[*lead, heads, dim]} on {device} expected, not {list(t.shape)}")
            strides = t.stride()
            if strides[-1] != 1 or (heads > 1 and strides[-2] != dim):
                raise ValueError(f"{what}: adjacent heads expected")
            distances.append(self._distance(strides, lead, heads * dim, what))
        Hv, g = self.Hv, log_decay.shape
        if log_decay.dtype != torch.float32 or log_decay.device != device or (g != (Hv,) and g != (*lead, Hv)) or \
                not _dense_rows(log_decay):
            raise ValueError(f"log_decay: f32 [{Hv}] or {[*lead, Hv]} on {device}")
        distances.append(self._distance(log_decay.stride(), lead, Hv, "log_decay") if len(g) > 1 else 0)
        if out is None:
            out = _empty(v.shape, torch.bfloat16, device, stream)
        elif out.shape != v.shape or out.dtype != torch.bfloat16 or not out.is_contiguous() or out.device != device:
            raise ValueError(f"out: contiguous bf16 {list(v.shape)} on {device}")
        return gdn.make_decay_tokens(q, k, v, log_decay, out, *distances), out

    def _check_slots(self, slot_idx, n):
        if slot_idx.dtype != torch.int32 or slot_idx.shape != (n,) or not _dense_rows(slot_idx) or \
                slot_idx.device != self.device:
            raise ValueError(f"slot_idx: contiguous int32 [{n}] on {self.device}")

    def step(self, slot_idx, q, k, v, log_decay, out=None, stream=None):
        """A token for each row, q and k bf16 [rows][num_k_heads][dk], v [rows][num_v_heads][dv]; or T of them,
        [rows][T][heads][dim].  log_decay f32 [num_v_heads], or one of each token.  slot_idx int32 [rows], -1:
        padding.  Returns out, of v's shape."""
        lead = tuple(v.shape[:-2])
        if len(lead) not in (1, 2):
            raise ValueError("v: [rows][num_v_heads][dv] or [rows][T][num_v_heads][dv]")
        self._check_slots(slot_idx, lead[0])
        tokens, out = self._tokens(lead, q, k, v, log_decay, out, stream)
        if lead[0]:
            gdn.gdn_decay_step(self.c, tokens, slot_idx, lead[1] if len(lead) == 2 else 1, stream)
        return out

    def workspace(self, num_seqs: int, total_tokens: int, stream=None) -> torch.Tensor:
        """The prefill's workspace on this stream: calls on one stream share it, a call that is captured in a CUDA
        graph gets memory of the graph's own."""
        with gdn.on_stream(stream):
            current = gdn.stream_handle()
            need = gdn.gdn_decay_prefill_workspace_bytes(self.c, num_seqs, total_tokens)
            if need == 0:
                raise ValueError("unsupported geometry")
            if torch.cuda.is_current_stream_capturing():
                return torch.empty(need, dtype=torch.uint8, device=self.device)
            ws = self._ws.get(current)
            if ws is None or ws.numel() < need:
                ws = self._ws[current] = torch.empty(need, dtype=torch.uint8, device=self.device)
            return ws

    def prefill(self, cu_seqlens, slot_idx, has_init, q, k, v, log_decay, out=None, stream=None):
        """Packed prompts: sequence n is tokens cu_seqlens[n] .. cu_seqlens[n + 1] of q, k [tokens][num_k_heads][dk]
        and v [tokens][num_v_heads][dv], and continues its slot's state where has_init[n] (uint8; None: none does)."""
        n = slot_idx.shape[0]
        self._check_slots(slot_idx, n)
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.shape != (n + 1,) or not _dense_rows(cu_seqlens) or \
                cu_seqlens.device != self.device:
            raise ValueError(f"cu_seqlens: contiguous int32 [{n + 1}] on {self.device}")
        if has_init is not None and (has_init.dtype not in (torch.uint8, torch.bool) or has_init.shape != (n,) or
                                     not _dense_rows(has_init) or has_init.device != self.device):
            raise ValueError(f"has_init: contiguous uint8 [{n}] on {self.device}")
        if v.dim() != 3:
            raise ValueError("v: [tokens][num_v_heads][dv]")
        if n == 0 and v.shape[0]:
            raise ValueError("tokens, but no sequence that they are in")
        tokens, out = self._tokens(tuple(v.shape[:1]), q, k, v, log_decay, out, stream)
        if n:
            gdn.gdn_decay_prefill(self.c, tokens, cu_seqlens, slot_idx, has_init, v.shape[0],
                                  self.workspace(n, v.shape[0], stream), stream)
        return out


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

    def append_rotated(self, batch: KVBatch, rotary: Rotary, q, k, v, q_norm=None, k_norm=None, eps=1e-6,
                       weight_offset=0.0, positions=None, q_out=None, stream=None):
        """append() of keys that are normed (k_norm: bf16 [head_dim]) and turned on the way, beside queries
        [total_tokens][num_q_heads][head_dim] (or None): returns these, normed and turned.  positions: device
        int32 [total_tokens]; None: the tokens' places in the cache."""
        for t, what in ((k, "k"), (v, "v")):
            shape, stride = self._check(t, batch, what)
            if shape[1] != self.num_kv_heads or (stride[1] != self.head_dim and self.num_kv_heads > 1):
                raise ValueError(f"{what}: {self.num_kv_heads} adjacent heads expected")
        device = self.device
        if q is not None:
            shape, _ = self._check(q, batch, "q")
            if q_out is None:
                q_out = _empty(shape, torch.bfloat16, device, stream)
            elif q_out.shape != shape or q_out.dtype != torch.bfloat16 or not q_out.is_contiguous() or q_out.device != device:
                raise ValueError("q_out: contiguous bf16 with the shape of q, on the cache's device")
        elif q_out is not None:
            raise ValueError("q_out without q")
        for t, what in ((q_norm, "q_norm"), (k_norm, "k_norm")):
            if t is not None and (t.shape != (self.head_dim,) or t.dtype != torch.bfloat16 or not _dense_rows(t) or
                                  t.device != device):
                raise ValueError(f"{what}: contiguous bf16 [{self.head_dim}] on the cache's device")
        if positions is not None and (positions.shape != (batch.total_tokens,) or positions.dtype != torch.int32 or
                                      not _dense_rows(positions) or positions.device != device):
            raise ValueError("positions: contiguous int32 [total_tokens] on the cache's device")
        if rotary.device != device:
            raise ValueError(f"the rotation is on {rotary.device}, the cache on {device}")
        if rotary.rot_dim > self.head_dim or rotary.rot_dim % 16:
            raise ValueError(f"a rotated part of {self.head_dim} elements at most, a multiple of 16, expected")
        if batch.total_tokens:
            gdn.gdn_kv_append_rotated(self.c, batch.c, rotary.c, gdn.make_head_prep(q_norm, k_norm, weight_offset, eps, positions),
                                      q, q_out, k, v, stream)
        return q_out

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
