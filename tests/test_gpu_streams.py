"""Calls on a stream that is not the current one, which lags behind while the current stream's
allocations go on."""
import pytest
import torch

import paged_ref as ref
from gated_deltanet_linear_09_gb300 import hybrid, runtime

pytestmark = pytest.mark.gpu


@pytest.fixture
def late():
    """A stream whose next work starts some milliseconds from now."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    return s


def _overwrite(shapes):
    """New tensors of the current stream, in whatever memory it thinks free."""
    for _ in range(4):
        for shape, dtype in shapes:
            torch.full(shape, 7, dtype=dtype, device="cuda")


def test_outputs_of_a_late_stream(late):
    case = ref.Case([3, 1], [200, 90], 2, 64, 16, True, seed=61)
    cache, b = case.filled_cache(runtime), case.device_batch(runtime)
    q = torch.randn((case.tokens, 8, 64), device="cuda").to(torch.bfloat16)
    x, w = torch.randn((512, 256), device="cuda"), torch.randn(256, device="cuda")
    want = [*(t for t in runtime.rms_norm(x, w, residual=x, quant="block")), *cache.read(b), cache.attend(b, q)]
    late.wait_stream(torch.cuda.current_stream())
    got = []
    for call in (lambda: runtime.rms_norm(x, w, residual=x, quant="block", stream=late), lambda: cache.read(b, stream=late),
                 lambda: (cache.attend(b, q, stream=late),)):
        out = call()
        with torch.cuda.stream(late):
            got += [t.clone() for t in out]
        shapes = [(t.shape, torch.uint8 if t.element_size() == 1 else t.dtype) for t in out]
        del out                         # the late stream has yet to write and copy it
        _overwrite(shapes)
    late.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_a_layer_on_a_late_stream(late):
    """With a rotation, whose tensors are torch's: the same bits as on the current stream."""
    n, hidden, new = 4, 128, [9, 1, 30, 4]
    w = hybrid.attention_weights(hidden, 4, 2, 64, 62)
    cu = [sum(new[:i]) for i in range(n + 1)]
    table = torch.arange(n * 2, dtype=torch.int32, device="cuda").view(n, 2)
    batch = runtime.KVBatch(torch.tensor(cu, dtype=torch.int32, device="cuda"),
                            torch.tensor(new, dtype=torch.int32, device="cuda"), table, cu[-1], max(new))
    x = torch.randn((cu[-1], hidden), device="cuda").to(torch.bfloat16)

    def rotate(q, k):
        return q * 2, (k.float() * 0.5 + 1).to(torch.bfloat16)

    def run(stream):
        cache = runtime.PagedKVCache(n * 2, 16, 2, 64)
        layer = hybrid.AttentionLayer(cache, 4, w)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        y = layer.forward(batch, x, rotate, stream=stream)
        if stream is not None:
            _overwrite([((cu[-1], c), torch.bfloat16) for c in (512, 256, 128, 128)])
            stream.synchronize()
        return y, cache.k_pages
    for a, b in zip(run(None), run(late)):
        assert torch.equal(a, b)


def test_graphs_replayed_beside_each_other():
    """Two graphs over one cache, captured on the same stream, replayed on two, and eager calls on the
    capture stream's workspace in between."""
    case = ref.Case([1] * 6, [900, 3000, 17, 2500, 1, 1200], 2, 128, 32, False, seed=63)
    cache, b = case.filled_cache(runtime), case.device_batch(runtime)
    qs = [torch.randn((6, 8, 128), device="cuda").to(torch.bfloat16) for _ in range(3)]
    want = [cache.attend(b, q).clone() for q in qs]
    outs, graphs = [torch.empty_like(q) for q in qs], []
    capture = torch.cuda.Stream()
    capture.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(capture):
        cache.attend(b, qs[2], out=outs[2])
    torch.cuda.synchronize()
    for q, o in zip(qs[:2], outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=capture):
            for _ in range(5):
                cache.attend(b, q, out=o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(capture):
            cache.attend(b, qs[2], out=outs[2])
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
