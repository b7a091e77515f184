"""Thin ctypes binding of libgdn.so (the C ABI declared in include/gdn.h).

Argument marshalling only: every function passes device pointers (``tensor.data_ptr()``),
sizes and the current CUDA stream to the C entry point of the same name and raises on a
non-zero return code.  Every step of the computation runs in the library's CUDA kernels.
There is no fallback: if the library has not been built, or cannot be loaded, every call
raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

from . import build as _build

GDN_F32 = 0
GDN_BF16 = 1
GDN_MAX_COMPACT_PAIRS = 2048
GDN_STATUS_SLOT_RANGE = 1
GDN_STATUS_BAD_SEQLENS = 2
GDN_STATUS_TIMEOUT = 4
GDN_STATUS_PAGE_RANGE = 8
GDN_NORM_ACT = 0
GDN_NORM_E4M3_ROW = 1
GDN_NORM_E4M3_BLOCK = 2
GDN_MAX_NORM_WIDTH = 32768
GDN_KV_BF16 = 0
GDN_KV_E4M3 = 1
GDN_MAX_ROTARY_DIM = 1024
GDN_GATE_NONE = 0
GDN_GATE_SIGMOID = 1
GDN_GATE_SILU = 2

_CODES = {
    0: "GDN_OK", -1: "GDN_ERR_INVALID_ARG", -2: "GDN_ERR_UNSUPPORTED_SHAPE",
    -3: "GDN_ERR_HEAD_DIVISIBILITY", -4: "GDN_ERR_SLOT_RANGE", -5: "GDN_ERR_WORKSPACE_TOO_SMALL",
    -6: "GDN_ERR_OVERLAP", -7: "GDN_ERR_MISALIGNED", -8: "GDN_ERR_CUDA", -9: "GDN_ERR_TOO_LARGE",
}

# Every symbol include/gdn.h declares.
EXPORTED = ("gdn_state_slot_bytes", "gdn_conv1d_update", "gdn_decode_step", "gdn_decode_multi",
            "gdn_prefill_workspace_bytes", "gdn_prefill_chunked", "gdn_state_compact",
            "gdn_status_string", "gdn_prefill_chunked_noalloc", "gdn_decode_graphs_create",
            "gdn_decode_graphs_buffers", "gdn_decode_graphs_launch", "gdn_decode_graphs_destroy",
            "gdn_proj_packed_bytes", "gdn_proj_pack", "gdn_linear_bf16", "gdn_in_proj",
            "gdn_out_proj", "gdn_rms_norm", "gdn_kv_append", "gdn_kv_read",
            "gdn_paged_attention_workspace_bytes", "gdn_paged_attention", "gdn_rotary_apply",
            "gdn_kv_append_rotated", "gdn_block_norm", "gdn_decay_step",
            "gdn_decay_prefill_workspace_bytes", "gdn_decay_prefill")
GDN_MAX_DECODE_TOKENS = 8
GDN_MAX_GRAPH_BUCKETS = 16
GDN_NOALLOC_PREFILL_SCRATCH_BYTES = 64 << 20
GDN_MAX_PROJ_SEGMENTS = 4
GDN_PROJ_BLOCK_BYTES = 16384


class GdnError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed: {_CODES.get(code, code)} ({msg})")
        self.code = code


class gdn_dims(ctypes.Structure):
    _fields_ = [("num_k_heads", ctypes.c_int32), ("num_v_heads", ctypes.c_int32),
                ("head_k_dim", ctypes.c_int32), ("head_v_dim", ctypes.c_int32),
                ("conv_kernel", ctypes.c_int32), ("q_scale", ctypes.c_float),
                ("l2_eps", ctypes.c_float), ("norm_eps", ctypes.c_float)]


class gdn_weights(ctypes.Structure):
    _fields_ = [("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("conv_weight", ctypes.c_void_p), ("norm_weight", ctypes.c_void_p),
                ("act", ctypes.c_int)]


class gdn_proj_route(ctypes.Structure):
    _fields_ = [("nseg", ctypes.c_int32), ("start", ctypes.c_int32 * GDN_MAX_PROJ_SEGMENTS),
                ("ld", ctypes.c_int32 * GDN_MAX_PROJ_SEGMENTS),
                ("dst", ctypes.c_void_p * GDN_MAX_PROJ_SEGMENTS)]


class gdn_pool(ctypes.Structure):
    _fields_ = [("rec_state", ctypes.c_void_p), ("conv_state", ctypes.c_void_p),
                ("num_slots", ctypes.c_int32), ("status", ctypes.c_void_p)]


class gdn_kv_cache(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("type", ctypes.c_int), ("status", ctypes.c_void_p)]


class gdn_kv_batch(ctypes.Structure):
    _fields_ = [("cu_seqlens", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("num_seqs", ctypes.c_int32),
                ("total_tokens", ctypes.c_int32), ("table_ld", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("table_cols", ctypes.c_int32)]


class gdn_rotary(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class gdn_head_prep(ctypes.Structure):
    _fields_ = [("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("weight_offset", ctypes.c_float),
                ("eps", ctypes.c_float), ("positions", ctypes.c_void_p)]


class gdn_block_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "gate", "residual", "post", "pre", "channel_scale")] + \
               [(n, ctypes.c_int64) for n in ("x_ld", "gate_ld", "residual_ld")] + \
               [("total", ctypes.c_void_p), ("y", ctypes.c_void_p)] + \
               [(n, ctypes.c_float) for n in ("scale", "weight_offset", "eps")] + \
               [("group", ctypes.c_int32), ("gate_act", ctypes.c_int)]


class gdn_decay_layer(ctypes.Structure):
    _fields_ = [("state", ctypes.c_void_p), ("num_slots", ctypes.c_int32), ("num_k_heads", ctypes.c_int32),
                ("num_v_heads", ctypes.c_int32), ("head_k_dim", ctypes.c_int32), ("head_v_dim", ctypes.c_int32),
                ("scale", ctypes.c_float), ("status", ctypes.c_void_p)]


class gdn_decay_tokens(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_ld", ctypes.c_int64),
                ("k_ld", ctypes.c_int64), ("v_ld", ctypes.c_int64), ("log_decay", ctypes.c_void_p),
                ("decay_ld", ctypes.c_int64), ("out", ctypes.c_void_p)]


_lib = None
_P = ctypes.c_void_p
_I32 = ctypes.c_int32


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False):
    """Load libgdn.so (optionally building it first).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if build_if_missing:
        path = _build.build()
    if not os.path.exists(path):
        raise RuntimeError(f"libgdn.so is not built ({path}); run __graft_entry__.build() or "
                           "python -m gated_deltanet_linear_09_gb300.build")
    lib = ctypes.CDLL(path)
    lib.gdn_state_slot_bytes.restype = ctypes.c_size_t
    lib.gdn_state_slot_bytes.argtypes = [_P, ctypes.c_int]
    lib.gdn_conv1d_update.restype = ctypes.c_int
    lib.gdn_conv1d_update.argtypes = [_P, _P, _P, _P, _I32, _P, _P, _P]
    lib.gdn_decode_step.restype = ctypes.c_int
    lib.gdn_decode_step.argtypes = [_P, _P, _P, _P, _I32, _P, _P, _P, _P, _P, _P]
    lib.gdn_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_decode_multi.argtypes = [_P, _P, _P, _P, _I32, _I32, _P, _P, _P, _P, _P, _P]
    lib.gdn_decode_multi.restype = ctypes.c_int
    lib.gdn_decode_graphs_create.argtypes = [_P, _P, _P, _P, _I32, _P]
    lib.gdn_decode_graphs_create.restype = ctypes.c_int
    lib.gdn_decode_graphs_buffers.argtypes = [_P] + [_P] * 7
    lib.gdn_decode_graphs_buffers.restype = ctypes.c_int
    lib.gdn_decode_graphs_launch.argtypes = [_P, _I32, _P]
    lib.gdn_decode_graphs_launch.restype = ctypes.c_int
    lib.gdn_decode_graphs_destroy.argtypes = [_P]
    lib.gdn_decode_graphs_destroy.restype = None
    lib.gdn_prefill_workspace_bytes.argtypes = [_P, _I32, _I32]
    lib.gdn_prefill_chunked.restype = ctypes.c_int
    lib.gdn_prefill_chunked.argtypes = [_P, _P, _P, _P, _P, _P, _I32, _I32, _P, _P, _P, _P, _P,
                                        _P, ctypes.c_size_t, _P]
    lib.gdn_prefill_chunked_noalloc.restype = ctypes.c_int
    lib.gdn_prefill_chunked_noalloc.argtypes = [_P, _P, _P, _P, _P, _P, _I32, _I32, _P, _P, _P, _P,
                                                _P, _P]
    lib.gdn_state_compact.restype = ctypes.c_int
    lib.gdn_state_compact.argtypes = [_P, ctypes.c_int, _P, _P, _P, _I32, _P]
    lib.gdn_proj_packed_bytes.restype = ctypes.c_size_t
    lib.gdn_proj_packed_bytes.argtypes = [_I32, _I32]
    lib.gdn_proj_pack.restype = ctypes.c_int
    lib.gdn_proj_pack.argtypes = [_P, _I32, _I32, _P, ctypes.c_size_t, _P]
    lib.gdn_linear_bf16.restype = ctypes.c_int
    lib.gdn_linear_bf16.argtypes = [_P, _P, _I32, _I32, _I32, _P, _I32, _P, _P]
    lib.gdn_in_proj.restype = ctypes.c_int
    lib.gdn_in_proj.argtypes = [_P, _P, _P, _I32, _I32, _P, _P, _P, _P, _P, _P]
    lib.gdn_out_proj.restype = ctypes.c_int
    lib.gdn_out_proj.argtypes = [_P, _P, _P, _I32, _I32, _P, _P, _P]
    i64, f32 = ctypes.c_int64, ctypes.c_float
    lib.gdn_rms_norm.restype = ctypes.c_int
    lib.gdn_rms_norm.argtypes = [_P, i64, _P, i64, _P, f32, f32, _I32, _I32, ctypes.c_int,
                                 ctypes.c_int, _P, _P, _P, _P]
    lib.gdn_kv_append.restype = ctypes.c_int
    lib.gdn_kv_append.argtypes = [_P, _P, _P, i64, _P, i64, _P]
    lib.gdn_kv_read.restype = ctypes.c_int
    lib.gdn_kv_read.argtypes = [_P, _P, _P, _P, _P]
    lib.gdn_paged_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_paged_attention_workspace_bytes.argtypes = [_P, _I32]
    lib.gdn_paged_attention.restype = ctypes.c_int
    lib.gdn_paged_attention.argtypes = [_P, _P, _I32, _P, i64, i64, _P, i64, i64, f32, _P, _P,
                                        ctypes.c_size_t, _P]
    lib.gdn_rotary_apply.restype = ctypes.c_int
    lib.gdn_rotary_apply.argtypes = [_P, _P, _I32, _I32, ctypes.c_int, _P, i64, i64, _I32, _P, _P, i64, i64,
                                     _I32, _P, _P]
    lib.gdn_kv_append_rotated.restype = ctypes.c_int
    lib.gdn_kv_append_rotated.argtypes = [_P, _P, _P, _P, _P, i64, i64, _I32, _P, _P, i64, _P, i64, _P]
    lib.gdn_block_norm.restype = ctypes.c_int
    lib.gdn_block_norm.argtypes = [_P, _I32, _I32, ctypes.c_int, _P]
    lib.gdn_decay_step.restype = ctypes.c_int
    lib.gdn_decay_step.argtypes = [_P, _P, _P, _I32, _I32, _P]
    lib.gdn_decay_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_decay_prefill_workspace_bytes.argtypes = [_P, _I32, _I32]
    lib.gdn_decay_prefill.restype = ctypes.c_int
    lib.gdn_decay_prefill.argtypes = [_P, _P, _P, _P, _P, _I32, _I32, _P, ctypes.c_size_t, _P]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_status_string.argtypes = [ctypes.c_int]
    _lib = lib
    return lib


def _check(fn: str, rc: int):
    if rc != 0:
        raise GdnError(fn, rc, load().gdn_status_string(rc).decode())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# The current stream's handle without building a Stream object (2.8 us of a 5 us call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _get_device is not None:
            return _raw_stream(_get_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def stream_handle(stream=None) -> int:
    """The cudaStream_t of a torch stream (None: the current one)."""
    return _stream(stream)


def on_stream(stream=None):
    """A context in which this stream (None, a torch stream or a cudaStream_t) is the current one, so
    that memory allocated in it is the stream's."""
    if stream is None or _stream(stream) == _stream(None):
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def act_code(dtype) -> int:
    if dtype == torch.bfloat16:
        return GDN_BF16
    if dtype == torch.float32:
        return GDN_F32
    raise ValueError(f"unsupported activation dtype {dtype}")


def make_dims(Hk, Hv, dk, dv, K=4, q_scale=0.0, l2_eps=1e-6, norm_eps=1e-6) -> gdn_dims:
    return gdn_dims(Hk, Hv, dk, dv, K, q_scale, l2_eps, norm_eps)


def make_weights(A_log, dt_bias, conv_weight, norm_weight) -> gdn_weights:
    return gdn_weights(_ptr(A_log), _ptr(dt_bias), _ptr(conv_weight), _ptr(norm_weight),
                       act_code(conv_weight.dtype))


def make_pool(rec_state, conv_state, status=None) -> gdn_pool:
    return gdn_pool(_ptr(rec_state), _ptr(conv_state), rec_state.shape[0], _ptr(status))


# ---------------------------------------------------------------- the C entry points

def gdn_state_slot_bytes(dims: gdn_dims, act: int) -> int:
    return int(load().gdn_state_slot_bytes(ctypes.byref(dims), act))


def gdn_conv1d_update(dims, weights, pool, slot_idx, qkv_in, qkv_out, stream=None):
    B = qkv_in.shape[0] if qkv_in is not None else 0
    _check("gdn_conv1d_update", load().gdn_conv1d_update(
        ctypes.byref(dims), ctypes.byref(weights), ctypes.byref(pool), _ptr(slot_idx), B,
        _ptr(qkv_in), _ptr(qkv_out), _stream(stream)))


def gdn_decode_step(dims, weights, pool, slot_idx, qkv, z, a, b, out, stream=None):
    B = slot_idx.shape[0]
    _check("gdn_decode_step", load().gdn_decode_step(
        ctypes.byref(dims), ctypes.byref(weights), ctypes.byref(pool), _ptr(slot_idx), B,
        _ptr(qkv), _ptr(z), _ptr(a), _ptr(b), _ptr(out), _stream(stream)))


def gdn_decode_multi(dims, weights, pool, slot_idx, qkv, z, a, b, out, stream=None):
    """T tokens per row: qkv [B][T][Cqkv], z/out [B][T][Hv*dv], a/b [B][T][Hv]."""
    B, T = int(qkv.shape[0]), int(qkv.shape[1])
    _check("gdn_decode_multi", load().gdn_decode_multi(
        ctypes.byref(dims), ctypes.byref(weights), ctypes.byref(pool), _ptr(slot_idx), B, T,
        _ptr(qkv), _ptr(z), _ptr(a), _ptr(b), _ptr(out), _stream(stream)))


def gdn_decode_graphs_create(dims, weights, pool, buckets) -> int:
    """Returns the object handle (an address)."""
    arr = (ctypes.c_int32 * len(buckets))(*[int(x) for x in buckets])
    h = ctypes.c_void_p()
    _check("gdn_decode_graphs_create", load().gdn_decode_graphs_create(
        ctypes.byref(dims), ctypes.byref(weights), ctypes.byref(pool), arr, len(buckets),
        ctypes.byref(h)))
    return h.value


def gdn_decode_graphs_buffers(handle) -> dict:
    """Device addresses of the static buffers and the largest bucket."""
    ptrs = [ctypes.c_void_p() for _ in range(6)]
    mb = ctypes.c_int32()
    _check("gdn_decode_graphs_buffers", load().gdn_decode_graphs_buffers(
        handle, *[ctypes.byref(p) for p in ptrs], ctypes.byref(mb)))
    d = dict(zip(("slot_idx", "qkv", "z", "a", "b", "out"), (p.value for p in ptrs)))
    d["max_batch"] = mb.value
    return d


def gdn_decode_graphs_launch(handle, B: int, stream=None):
    _check("gdn_decode_graphs_launch", load().gdn_decode_graphs_launch(handle, B, _stream(stream)))


def gdn_decode_graphs_destroy(handle):
    load().gdn_decode_graphs_destroy(handle)


def gdn_prefill_workspace_bytes(dims, num_seqs: int, total_tokens: int) -> int:
    return int(load().gdn_prefill_workspace_bytes(ctypes.byref(dims), num_seqs, total_tokens))


def gdn_prefill_chunked(dims, weights, pool, cu_seqlens, slot_idx, has_initial_state, num_seqs,
                        total_tokens, qkv, z, a, b, out, workspace, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("gdn_prefill_chunked", load().gdn_prefill_chunked(
        ctypes.byref(dims), ctypes.byref(weights), ctypes.byref(pool), _ptr(cu_seqlens),
        _ptr(slot_idx), _ptr(has_initial_state), num_seqs, total_tokens, _ptr(qkv), _ptr(z),
        _ptr(a), _ptr(b), _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)))


def gdn_prefill_chunked_noalloc(dims, weights, pool, cu_seqlens, slot_idx, has_initial_state,
                                num_seqs, total_tokens, qkv, z, a, b, out, stream=None):
    """Prefill whose scratch is the library's fixed device array: allocates nothing."""
    _check("gdn_prefill_chunked_noalloc", load().gdn_prefill_chunked_noalloc(
        ctypes.byref(dims), ctypes.byref(weights), ctypes.byref(pool), _ptr(cu_seqlens),
        _ptr(slot_idx), _ptr(has_initial_state), num_seqs, total_tokens, _ptr(qkv), _ptr(z),
        _ptr(a), _ptr(b), _ptr(out), _stream(stream)))


def gdn_state_compact(dims, act: int, pool, src_slots, dst_slots, stream=None):
    src = (ctypes.c_int32 * len(src_slots))(*[int(x) for x in src_slots])
    dst = (ctypes.c_int32 * len(dst_slots))(*[int(x) for x in dst_slots])
    if len(src_slots) != len(dst_slots):
        raise ValueError("src_slots and dst_slots differ in length")
    _check("gdn_state_compact", load().gdn_state_compact(
        ctypes.byref(dims), act, ctypes.byref(pool), src, dst, len(src_slots), _stream(stream)))


def make_route(segments) -> gdn_proj_route:
    """segments: [(start, ld, dst tensor or address), ...] in increasing start order."""
    r = gdn_proj_route()
    r.nseg = len(segments)
    for i, (start, ld, dst) in enumerate(segments):
        r.start[i] = int(start)
        r.ld[i] = int(ld)
        r.dst[i] = _ptr(dst)
    return r


def gdn_proj_packed_bytes(N: int, K: int) -> int:
    return int(load().gdn_proj_packed_bytes(int(N), int(K)))


def gdn_proj_pack(w, packed, stream=None):
    """Packs a bf16 linear weight w [N][K] into the tile layout (packed: a uint8 device tensor)."""
    N, K = int(w.shape[0]), int(w.shape[1])
    _check("gdn_proj_pack", load().gdn_proj_pack(
        _ptr(w), N, K, _ptr(packed), packed.numel() * packed.element_size(), _stream(stream)))


def gdn_linear_bf16(x, w_packed, N: int, route: gdn_proj_route, k_split: int = 0, status=None,
                    stream=None):
    """y = x w^T (bf16, f32 sums): x [M][K], w packed from [N][K]; outputs go where route says."""
    M, K = int(x.shape[0]), int(x.shape[1])
    _check("gdn_linear_bf16", load().gdn_linear_bf16(
        _ptr(x), _ptr(w_packed), M, int(N), K, ctypes.byref(route), int(k_split), _ptr(status),
        _stream(stream)))


def gdn_in_proj(dims, hidden, w_in_packed, qkv, z, b, a, status=None, stream=None):
    """hidden [rows][H], packed w_in [Cqkv + Hv*dv + 2*Hv][H] -> qkv, z, b, a (step layouts)."""
    rows, H = int(hidden.shape[0]), int(hidden.shape[1])
    _check("gdn_in_proj", load().gdn_in_proj(
        ctypes.byref(dims), _ptr(hidden), _ptr(w_in_packed), rows, H, _ptr(qkv), _ptr(z),
        _ptr(b), _ptr(a), _ptr(status), _stream(stream)))


def gdn_out_proj(dims, out, w_out_packed, y, status=None, stream=None):
    """out [rows][Hv*dv], packed w_out [H][Hv*dv] -> y [rows][H] (bf16)."""
    rows, H = int(out.shape[0]), int(y.shape[1])
    _check("gdn_out_proj", load().gdn_out_proj(
        ctypes.byref(dims), _ptr(out), _ptr(w_out_packed), rows, H, _ptr(y), _ptr(status),
        _stream(stream)))


def _on_host(fn: str):
    """The library takes addresses as they are: one of host memory would end in a GPU fault."""
    raise ValueError(f"{fn}: its tensors are not on a GPU")


def make_kv_cache(k_pages, v_pages, k_scales=None, v_scales=None, status=None) -> gdn_kv_cache:
    """Pages [num_pages][num_kv_heads][page_size][head_dim] (bf16 or float8_e4m3fn) as a struct."""
    np_, heads, page, dim = (int(x) for x in k_pages.shape)
    q8 = k_pages.dtype == torch.float8_e4m3fn
    if not q8 and k_pages.dtype != torch.bfloat16:
        raise ValueError(f"unsupported cache dtype {k_pages.dtype}")
    return gdn_kv_cache(_ptr(k_pages), _ptr(v_pages), _ptr(k_scales), _ptr(v_scales), np_, page,
                        heads, dim, GDN_KV_E4M3 if q8 else GDN_KV_BF16, _ptr(status))


def make_kv_batch(cu_seqlens, kv_lens, block_table, total_tokens: int, max_tokens: int = 0) -> gdn_kv_batch:
    """Device int32 tensors: cu_seqlens [n + 1], kv_lens [n], block_table [n][table_ld] (rows may be
    strided, or all the same one)."""
    cols = int(block_table.shape[1])
    ld = int(block_table.stride(0)) if block_table.shape[0] > 1 and cols else cols
    return gdn_kv_batch(_ptr(cu_seqlens), _ptr(kv_lens), _ptr(block_table), int(kv_lens.shape[0]),
                        int(total_tokens), ld, int(max_tokens), cols)


def gdn_rms_norm(x, weight, y, residual=None, sum_out=None, scales=None, weight_offset=0.0, eps=1e-6,
                 out_kind=GDN_NORM_ACT, stream=None):
    """x, residual [rows][n] (rows may be strided), y / sum_out dense [rows][n], scales f32."""
    rows, n = x.shape
    if not x.is_cuda:
        _on_host("gdn_rms_norm")
    rc = load().gdn_rms_norm(
        x.data_ptr(), x.stride(0) if rows > 1 else n, _ptr(residual),
        0 if residual is None else residual.stride(0) if rows > 1 else n, weight.data_ptr(),
        weight_offset, eps, rows, n, act_code(x.dtype), out_kind, _ptr(sum_out), y.data_ptr(),
        _ptr(scales), _stream(stream))
    if rc:
        _check("gdn_rms_norm", rc)


def gdn_kv_append(cache, batch, k, v, stream=None):
    """k, v: bf16 [tokens][heads][dim], token rows may be strided."""
    if not k.is_cuda:
        _on_host("gdn_kv_append")
    tokens, heads, dim = k.shape
    if tokens == 1:                   # the stride of a dimension of size one says nothing
        k_ld = v_ld = heads * dim
    else:
        k_ld, v_ld = k.stride()[0], v.stride()[0]
    rc = load().gdn_kv_append(ctypes.byref(cache), ctypes.byref(batch), k.data_ptr(), k_ld, v.data_ptr(),
                              v_ld, _stream(stream))
    if rc:
        _check("gdn_kv_append", rc)


def gdn_kv_read(cache, batch, k, v, stream=None):
    """k, v: dense bf16 [tokens][heads][dim] outputs."""
    if not k.is_cuda:
        _on_host("gdn_kv_read")
    _check("gdn_kv_read", load().gdn_kv_read(
        ctypes.byref(cache), ctypes.byref(batch), k.data_ptr(), v.data_ptr(), _stream(stream)))


def gdn_paged_attention_workspace_bytes(cache, num_q_heads: int) -> int:
    return int(load().gdn_paged_attention_workspace_bytes(ctypes.byref(cache), int(num_q_heads)))


def gdn_paged_attention(cache, batch, q, out, workspace, gate=None, scale=0.0, stream=None):
    """q, gate: bf16 [tokens][heads][dim] (tokens and heads may be strided), out dense, workspace
    uint8."""
    if not q.is_cuda:
        _on_host("gdn_paged_attention")
    tokens, heads, dim = q.shape
    q_ld, q_head_ld, _ = q.stride()
    g_ld, g_head_ld, _ = (0, 0, 0) if gate is None else gate.stride()
    if tokens == 1:                   # the stride of a dimension of size one says nothing
        q_ld = g_ld = heads * dim
    if heads == 1:
        q_head_ld = g_head_ld = dim
    rc = load().gdn_paged_attention(
        ctypes.byref(cache), ctypes.byref(batch), heads, q.data_ptr(), q_ld, q_head_ld,
        None if gate is None else gate.data_ptr(), g_ld, g_head_ld, scale, out.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _stream(stream))
    if rc:
        _check("gdn_paged_attention", rc)


def make_rotary(turns, rot_dim: int, interleaved: bool = False, scale: float = 1.0) -> gdn_rotary:
    """turns: device int64 [rot_dim / 2], each pair's turns a position in units of 2^-64 (modulo 2^64)."""
    return gdn_rotary(_ptr(turns), int(rot_dim), int(bool(interleaved)), float(scale))


def _head_strides(t):
    """(token distance, head distance) of [tokens][heads][dim]; of dimensions of size one, the dense ones."""
    tokens, heads, dim = t.shape
    ld, head_ld, _ = t.stride()
    if heads == 1:
        head_ld = dim
    if tokens == 1:
        ld = max(heads * dim, (heads - 1) * head_ld + dim)
        ld += -ld % 8 if head_ld % 8 == 0 and dim % 8 == 0 else 0
    return ld, head_ld


def gdn_rotary_apply(rotary, positions, q=None, q_out=None, k=None, k_out=None, stream=None):
    """q, k: [tokens][heads][dim] (tokens and heads may be strided), outputs dense."""
    t = q if q is not None else k
    if not t.is_cuda:
        _on_host("gdn_rotary_apply")
    args = []
    for x, y in ((q, q_out), (k, k_out)):
        args += [None, 0, 0, 0, None] if x is None else [x.data_ptr(), *_head_strides(x), x.shape[1], y.data_ptr()]
    rc = load().gdn_rotary_apply(ctypes.byref(rotary), positions.data_ptr(), t.shape[0], t.shape[2], act_code(t.dtype),
                                 *args, _stream(stream))
    if rc:
        _check("gdn_rotary_apply", rc)


def make_head_prep(q_norm=None, k_norm=None, weight_offset=0.0, eps=1e-6, positions=None) -> gdn_head_prep:
    return gdn_head_prep(_ptr(q_norm), _ptr(k_norm), float(weight_offset), float(eps), _ptr(positions))


def gdn_kv_append_rotated(cache, batch, rotary, prep, q, q_out, k, v, stream=None):
    """q: bf16 [tokens][heads][dim] (tokens and heads may be strided; None: none), q_out dense; k, v as for
    gdn_kv_append."""
    if not k.is_cuda:
        _on_host("gdn_kv_append_rotated")
    tokens, heads, dim = k.shape
    if tokens == 1:                   # the stride of a dimension of size one says nothing
        k_ld = v_ld = heads * dim
    else:
        k_ld, v_ld = k.stride()[0], v.stride()[0]
    q_args = (None, 0, 0, 0, None) if q is None else (q.data_ptr(), *_head_strides(q), q.shape[1], q_out.data_ptr())
    rc = load().gdn_kv_append_rotated(ctypes.byref(cache), ctypes.byref(batch), ctypes.byref(rotary), ctypes.byref(prep),
                                      *q_args, k.data_ptr(), k_ld, v.data_ptr(), v_ld, _stream(stream))
    if rc:
        _check("gdn_kv_append_rotated", rc)


def gdn_block_norm(x, total=None, y=None, post=None, gate=None, gate_act=GDN_GATE_NONE, residual=None, pre=None,
                   channel_scale=None, scale=1.0, weight_offset=0.0, eps=1e-6, group=0, stream=None):
    """x, gate, residual [rows][n] (rows may be strided), total and y dense; group 0: the row."""
    if not x.is_cuda:
        _on_host("gdn_block_norm")
    rows, n = x.shape
    x_ld, gate_ld, residual_ld = (0 if t is None else t.stride(0) if rows > 1 else n for t in (x, gate, residual))
    a = gdn_block_args(x.data_ptr(), _ptr(gate), _ptr(residual), _ptr(post), _ptr(pre), _ptr(channel_scale), x_ld, gate_ld,
                       residual_ld, _ptr(total), _ptr(y), scale, weight_offset, eps, group or n, gate_act)
    rc = load().gdn_block_norm(ctypes.byref(a), rows, n, act_code(x.dtype), _stream(stream))
    if rc:
        _check("gdn_block_norm", rc)


def make_decay_layer(state, num_k_heads: int, scale: float = 0.0, status=None) -> gdn_decay_layer:
    """state f32 [num_slots][num_v_heads][dk][dv]."""
    n, hv, dk, dv = (int(x) for x in state.shape)
    return gdn_decay_layer(_ptr(state), n, int(num_k_heads), hv, dk, dv, float(scale), _ptr(status))


def make_decay_tokens(q, k, v, log_decay, out, q_ld: int, k_ld: int, v_ld: int, decay_ld: int) -> gdn_decay_tokens:
    """q, k, v: bf16 tokens of adjacent heads, q_ld .. elements apart; log_decay f32 [heads] (decay_ld 0) or of
    each token; out dense."""
    return gdn_decay_tokens(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_ld, k_ld, v_ld, log_decay.data_ptr(), decay_ld,
                            out.data_ptr())


def gdn_decay_step(layer, tokens, slot_idx, T: int, stream=None):
    if not slot_idx.is_cuda:
        _on_host("gdn_decay_step")
    rc = load().gdn_decay_step(ctypes.byref(layer), ctypes.byref(tokens), slot_idx.data_ptr(), slot_idx.shape[0], T,
                               _stream(stream))
    if rc:
        _check("gdn_decay_step", rc)


def gdn_decay_prefill_workspace_bytes(layer, num_seqs: int, total_tokens: int) -> int:
    return int(load().gdn_decay_prefill_workspace_bytes(ctypes.byref(layer), int(num_seqs), int(total_tokens)))


def gdn_decay_prefill(layer, tokens, cu_seqlens, slot_idx, has_initial_state, total_tokens: int, workspace, stream=None):
    if not slot_idx.is_cuda:
        _on_host("gdn_decay_prefill")
    rc = load().gdn_decay_prefill(ctypes.byref(layer), ctypes.byref(tokens), cu_seqlens.data_ptr(), slot_idx.data_ptr(),
                                  _ptr(has_initial_state), slot_idx.shape[0], total_tokens, workspace.data_ptr(),
                                  workspace.numel(), _stream(stream))
    if rc:
        _check("gdn_decay_prefill", rc)


def gdn_status_string(code: int) -> str:
    return load().gdn_status_string(code).decode()
