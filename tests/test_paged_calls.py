"""What the Python calls hand to the library, and which tensors they take (no GPU: nothing is launched)."""
import contextlib
import ctypes
import os
import subprocess
import types

import pytest
import torch

from gated_deltanet_linear_09_gb300 import build as gbuild
from gated_deltanet_linear_09_gb300 import gdn, hybrid, runtime


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_tables_carry_their_width():
    """A row of a table has its own number of entries, whatever the distance of the rows."""
    def batch(table):
        return runtime.KVBatch(ints(table.shape[0] + 1), ints(table.shape[0]), table, 4).c
    for table, ld, cols in ((ints(3, 5), 5, 5), (ints(3, 8)[:, 2:4], 8, 2), (ints(1, 6).expand(3, 6), 0, 6),
                            (ints(1, 8)[:, :3], 3, 3), (ints(3, 0), 0, 0)):
        b = batch(table)
        assert (b.table_ld, b.table_cols) == (ld, cols)
    assert gdn.gdn_kv_batch.table_cols.offset == gdn.gdn_kv_batch.max_tokens.offset + 4


def test_table_width_is_checked():
    gbuild.build()
    A = 0x10000
    cache = gdn.gdn_kv_cache(A, A, None, None, 4, 16, 2, 128, gdn.GDN_KV_BF16, None)

    def read(**kw):
        d = dict(cu_seqlens=A, kv_lens=A, block_table=A, num_seqs=1, total_tokens=1, table_ld=4, max_tokens=1)
        return gdn.load().gdn_kv_read(ctypes.byref(cache), ctypes.byref(gdn.gdn_kv_batch(**{**d, **kw})), A + 2, A, None)
    assert read(table_cols=-1) == -1
    assert read(table_ld=0, table_cols=3, block_table=None) == -1
    assert read(table_ld=0, table_cols=3) == -7                     # (on to the next check: k is misaligned)


class Streams:
    """Stands in for torch's streams: which one is current, and on which one each tensor was allocated."""

    def __init__(self, monkeypatch):
        self.current, self.allocated, self.launched = 0, [], []
        empty = torch.empty

        @contextlib.contextmanager
        def stream(s):
            before, self.current = self.current, s.cuda_stream
            yield
            self.current = before

        def recorded(*a, **kw):
            self.allocated.append(self.current)
            return empty(*a, **kw)
        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: types.SimpleNamespace(cuda_stream=handle))
        monkeypatch.setattr(torch, "empty", recorded)
        monkeypatch.setattr(gdn, "_stream", lambda s=None: self.current if s is None else s if isinstance(s, int) else s.cuda_stream)
        for name in gdn.EXPORTED:
            if hasattr(gdn, name) and not name.endswith("bytes"):
                monkeypatch.setattr(gdn, name, lambda *a, name=name: self.launched.append((name, a)))
        monkeypatch.setattr(gdn, "gdn_paged_attention_workspace_bytes", lambda *a: 512)
        self.capturing = False
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capturing)


@pytest.fixture
def streams(monkeypatch):
    return Streams(monkeypatch)


SIDE = types.SimpleNamespace(cuda_stream=7)


def test_outputs_belong_to_the_stream_that_writes_them(streams):
    """What a call on another stream allocates is that stream's memory, and the current stream stays."""
    bf = dict(dtype=torch.bfloat16)
    x, w = torch.zeros((4, 64), **bf), torch.zeros(64, **bf)
    cache = runtime.PagedKVCache(4, 16, 2, 64, device="cpu")
    batch = runtime.KVBatch(ints(3), ints(2), ints(2, 2), 4, 2)
    q = torch.zeros((4, 4, 64), **bf)
    calls = [lambda s: runtime.rms_norm(x, w, residual=x, stream=s), lambda s: runtime.rms_norm(x, w, quant="row", stream=s),
             lambda s: cache.read(batch, stream=s), lambda s: cache.attend(batch, q, stream=s),
             lambda s: cache.workspace(4, s)]
    for call in calls:
        for s, want in ((None, 0), (SIDE, 7), (types.SimpleNamespace(cuda_stream=0), 0)):
            cache._ws.clear()
            streams.allocated.clear()
            call(s)
            assert streams.allocated and set(streams.allocated) == {want} and streams.current == 0


def test_the_layer_runs_on_one_stream(streams):
    """Every allocation, launch and the rotation of a layer's call happen on the call's stream."""
    bf = dict(dtype=torch.bfloat16)
    cache = runtime.PagedKVCache(4, 16, 2, 64, device="cpu")
    layer = hybrid.AttentionLayer.__new__(hybrid.AttentionLayer)
    layer.cache, layer.Hq, layer.H, layer.D, layer.eps, layer.hidden = cache, 4, 2, 64, 1e-6, 32
    layer.w_in = layer.w_out = layer.status = None
    layer.q_norm = layer.k_norm = torch.zeros(64, **bf)
    batch = runtime.KVBatch(ints(3), ints(2), ints(2, 2), 3, 2)
    x, rotated = torch.zeros((3, 32), **bf), []

    def rotate(q, k):
        rotated.append(streams.current)
        return q, k
    for s, want in ((None, 0), (SIDE, 7)):
        streams.allocated.clear()
        streams.launched.clear()
        layer.forward(batch, x, rotate, stream=s)
        assert set(streams.allocated) == {want} and rotated.pop() == want and streams.current == 0
        assert [n for n, _ in streams.launched] == ["gdn_linear_bf16", "gdn_rms_norm", "gdn_rms_norm", "gdn_kv_append",
                                                    "gdn_paged_attention", "gdn_linear_bf16"]
        assert {a[-1] for n, a in streams.launched if isinstance(a[-1], (int, types.SimpleNamespace))} <= {want}


def test_workspaces_of_streams_and_graphs(streams):
    """One for each stream, whatever the number of query heads; a captured call's is the graph's alone."""
    cache = runtime.PagedKVCache(4, 16, 2, 64, device="cpu")
    here, side = cache.workspace(4), cache.workspace(4, SIDE)
    assert here is cache.workspace(8) and side is cache.workspace(2, SIDE) and here is not side
    streams.capturing = True
    a, b, c = cache.workspace(4), cache.workspace(4), cache.workspace(4, SIDE)
    assert len({t.data_ptr() for t in (here, side, a, b, c)}) == 5
    streams.capturing = False
    assert cache.workspace(4) is here and cache.workspace(4, SIDE) is side and len(cache._ws) == 2
    batch = runtime.KVBatch(ints(3), ints(2), ints(2, 2), 4, 2)
    q, used = torch.zeros((4, 4, 64), dtype=torch.bfloat16), []
    for streams.capturing in (False, True, True):
        streams.launched.clear()
        cache.attend(batch, q)
        used.append(streams.launched[0][1][4])
    assert used[0] is here and used[1] is not here and used[2] is not here


def test_kernel_attributes_are_set_on_every_device(tmp_path):
    """The guard that the launches share: once on each device, a failure not kept."""
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "once_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", gbuild.CSRC, "-o", exe,
                    os.path.join(here, "csrc", "once_check.cc")], check=True)
    assert subprocess.run([exe], capture_output=True, text=True).stdout == "ok\n"


def test_strides_of_single_elements_are_not_looked_at(streams):
    """One token, head, column or page: any stride is as good as the dense one."""
    bf = dict(dtype=torch.bfloat16)
    one = runtime.KVBatch(ints(2), ints(1), ints(1, 2), 1, 1)
    cache = runtime.PagedKVCache(4, 16, 2, 64, device="cpu")
    x = torch.zeros((2, 1, 64), **bf).transpose(0, 1)                    # head-major: strides 64, 64, 1
    cache.append(one, x, torch.zeros((1, 2, 64), **bf).as_strided((1, 2, 64), (8, 64, 1)))
    name, a = streams.launched[-1]
    assert name == "gdn_kv_append"
    single = runtime.PagedKVCache(4, 16, 1, 64, device="cpu")
    two = runtime.KVBatch(ints(2), ints(1), ints(1, 2), 2, 2)
    single.append(two, torch.zeros((2, 1, 64), **bf).as_strided((2, 1, 64), (64, 1, 1)), torch.zeros((2, 1, 64), **bf))
    runtime.rms_norm(torch.zeros((1, 5), **bf).t(), torch.zeros(2, **bf)[::2])
    runtime.KVBatch(ints(3), ints(2), ints(2, 4)[:, ::4], 2)
    with pytest.raises(ValueError):
        runtime.rms_norm(torch.zeros((4, 5), **bf).t(), torch.zeros(4, **bf))


def test_row_distances_handed_over(monkeypatch):
    """What the library sees of such tensors."""
    seen = {}

    class Gpu(torch.Tensor):
        is_cuda = True

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.update({name: a}) or 0
    monkeypatch.setattr(gdn, "load", lambda: Lib())
    monkeypatch.setattr(gdn, "_stream", lambda s: 0)
    c = gdn.gdn_kv_cache(num_kv_heads=2, head_dim=64)
    b = gdn.gdn_kv_batch()
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16).as_subclass(Gpu).transpose(0, 1)
    gdn.gdn_kv_append(c, b, x, x)
    assert seen["gdn_kv_append"][3] == seen["gdn_kv_append"][5] == 128
    two = torch.zeros((3, 400), dtype=torch.bfloat16).as_subclass(Gpu)[:, :128].view(3, 2, 64)
    gdn.gdn_kv_append(c, b, two, two)
    assert seen["gdn_kv_append"][3] == seen["gdn_kv_append"][5] == 400
    ws = torch.zeros(1, dtype=torch.uint8)
    gdn.gdn_paged_attention(c, b, x, x, ws, gate=x)
    assert seen["gdn_paged_attention"][4:6] == (128, 64) and seen["gdn_paged_attention"][7:9] == (128, 64)
    single = torch.zeros((3, 1, 64), dtype=torch.bfloat16).as_subclass(Gpu).as_strided((3, 1, 64), (64, 1, 1))
    gdn.gdn_paged_attention(c, b, single, single, ws)
    assert seen["gdn_paged_attention"][4:6] == (64, 64)
    gdn.gdn_paged_attention(c, b, two, two, ws)
    assert seen["gdn_paged_attention"][4:6] == (400, 64)


def test_tensors_of_other_devices_are_refused(streams):
    """Host memory, or memory of another device than the cache's, never reaches the library."""
    bf = dict(dtype=torch.bfloat16)

    def on(dev, *shape, **kw):
        return torch.zeros(shape, device=dev, **(kw or bf))
    cache = runtime.PagedKVCache(4, 16, 2, 64, device="cpu")
    batch = runtime.KVBatch(ints(3), ints(2), ints(2, 2), 3, 2)
    far = runtime.KVBatch(*(t.to("meta") for t in batch.tensors), 3, 2)
    t, m = on("cpu", 3, 2, 64), on("meta", 3, 2, 64)
    w8, u8 = torch.zeros(512, dtype=torch.uint8), dict(dtype=torch.uint8)
    refused = [
        lambda: runtime.KVBatch(ints(3).to("meta"), ints(2), ints(2, 2), 3), lambda: runtime.KVBatch(ints(3), ints(2), ints(2, 2).to("meta"), 3),
        lambda: runtime.KVBatch(ints(3, 1), ints(2), ints(2, 2), 3),
        lambda: runtime.PagedKVCache.over(cache.k_pages, cache.v_pages.to("meta")),
        lambda: cache.append(batch, t, m), lambda: cache.append(batch, m, t), lambda: cache.append(far, t, t),
        lambda: cache.read(far), lambda: cache.read(batch, m, t), lambda: cache.read(batch, t, m),
        lambda: cache.attend(batch, m), lambda: cache.attend(far, t), lambda: cache.attend(batch, t, gate=m), lambda: cache.attend(batch, t, out=m),
        lambda: cache.attend(batch, t, workspace=torch.zeros(1, **u8).expand(512)),
        lambda: cache.attend(batch, t, workspace=w8.view(torch.int32)), lambda: cache.attend(batch, t, workspace=w8.to("meta")),
        lambda: runtime.rms_norm(on("cpu", 2, 8), on("meta", 8)), lambda: runtime.rms_norm(on("meta", 2, 8), on("cpu", 8)),
        lambda: runtime.rms_norm(on("cpu", 2, 8), on("cpu", 8), residual=on("meta", 2, 8)),
        lambda: runtime.rms_norm(on("cpu", 2, 8), on("cpu", 8), quant="rows"),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError):
            call()
        assert not streams.launched, i
    cache.attend(batch, t, gate=t, out=t.clone(), workspace=w8)
    assert len(streams.launched) == 1


def test_host_memory_is_refused(monkeypatch):
    monkeypatch.setattr(gdn, "load", lambda: pytest.fail("the library was called"))
    x, ws = torch.zeros((2, 2, 64), dtype=torch.bfloat16), torch.zeros(8, dtype=torch.uint8)
    c, b = gdn.gdn_kv_cache(), gdn.gdn_kv_batch()
    for call in (lambda: gdn.gdn_rms_norm(x[0], x[0, 0], x[0]), lambda: gdn.gdn_kv_append(c, b, x, x),
                 lambda: gdn.gdn_kv_read(c, b, x, x), lambda: gdn.gdn_paged_attention(c, b, x, x, ws)):
        with pytest.raises(ValueError, match="not on a GPU"):
            call()


def test_heads_past_the_units_of_work_are_refused():
    """Groups so large that keys times heads leave 31 bits."""
    gbuild.build()
    A = 0x10000
    cache = gdn.gdn_kv_cache(A, A, None, None, 4, 16, 1, 128, gdn.GDN_KV_BF16, None)
    batch = gdn.gdn_kv_batch(A, A, A, 1, 1, 4, 1)

    def attend(heads, ws=A):
        return gdn.load().gdn_paged_attention(ctypes.byref(cache), ctypes.byref(batch), heads, A, 1 << 31, 128, None, 0, 0, 0.0, A,
                                              ws, 1 << 40, None)
    assert attend((1 << 20) + 1) == -9 and attend(1 << 25) == -9
    assert attend(1 << 20, ws=A + 16) == -7             # (on to the next check: the workspace is misaligned)
