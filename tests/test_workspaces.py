"""The workspaces that the binding caches: which calls share one, and how long it lives."""
import os
import weakref

import pytest

torch = pytest.importorskip("torch")
awq = pytest.importorskip("bit_weight_only_w4a16_amd.awq")


@pytest.fixture
def on_host(monkeypatch):
    """The cache with its buffers on the host, empty, and on stream 7."""
    if not os.path.exists(awq.LIB_PATH):
        pytest.skip("library not built")
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: real(*a, **kw))
    monkeypatch.setattr(awq, "_WS", {})
    monkeypatch.setattr(awq, "_stream", lambda device=None: 7)


def test_a_replaced_workspace_of_a_product_stays(on_host):
    """A graph may have been captured with it."""
    small = awq.workspace(300, 4096, 4096, "cuda:0")
    alive = weakref.ref(small)
    assert awq.workspace(64, 4096, 4096, "cuda:0") is small
    del small
    large = awq.workspace(8192, 4096, 4096, "cuda:0")
    assert large.numel() >= awq.awq_workspace_bytes(8192, 4096, 4096)
    assert alive() is not None and alive() is not large
    assert awq.workspace(300, 4096, 4096, "cuda:0") is large


@pytest.mark.gpu
@pytest.mark.parametrize("m", [40, 300])
def test_a_graph_of_a_layer_keeps_its_workspace(m):
    """A larger call after a layer with a tail was captured (split sums; X' and split sums):
    what is allocated then is not what the graph writes to."""
    g = torch.Generator().manual_seed(m)
    n, k = 264, 8192
    w = (torch.randn(n, k, generator=g) * 0.05).half().cuda()
    layer = awq.QuantLinear.from_weight(w, torch.randn(32, k, generator=g).half().cuda())
    x, r = torch.randn(m, k, generator=g).half().cuda(), torch.randn(m, n, generator=g).half().cuda()
    big = torch.randn(4096, k, generator=g).half().cuda()
    assert 0 < awq.awq_workspace_bytes(m, n, k) < awq.awq_workspace_bytes(4096, n, k)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        want = layer(x, act="silu", mul=r)
        graph = torch.cuda.CUDAGraph()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            out = layer(x, act="silu", mul=r)
        layer(big)
        others = [torch.full((1 << 20,), 77, dtype=torch.uint8, device="cuda") for _ in range(16)]
        for _ in range(3):
            out.zero_()
            graph.replay()
            stream.synchronize()
            assert torch.equal(out, want)
            assert all(bool((t == 77).all()) for t in others)
