"""The workspaces that the binding caches: which calls share one, and how long it lives."""
import os
import threading
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
    monkeypatch.setattr(awq, "_capturing", lambda index: False)


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


def test_every_captured_call_has_a_workspace_of_its_own(on_host, monkeypatch):
    eager = awq.scratch(100, 0)
    monkeypatch.setattr(awq, "_capturing", lambda index: True)
    first, second = awq.scratch(100, 0), awq.workspace(300, 4096, 4096, "cuda:0")
    assert len({t.data_ptr() for t in (eager, first, second)}) == 3
    assert awq.scratch(100, 0) is not first
    monkeypatch.setattr(awq, "_capturing", lambda index: False)
    assert awq.scratch(100, 0) is eager


def test_threads_on_one_stream_have_workspaces_of_their_own(on_host):
    """The launches of one call that uses a workspace may stand between those of another's."""
    inside, together = {}, threading.Barrier(2)

    def call(name):
        first = awq.scratch(100, 0)
        together.wait()   # (both threads live: their numbers differ)
        inside[name] = (first, awq.scratch(50, 0), awq.workspace(64, 4096, 4096, "cuda:0"))
        together.wait()

    threads = [threading.Thread(target=call, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert inside[i][0] is inside[i][1]
    assert len({t.data_ptr() for i in range(2) for t in inside[i]}) == 4


@pytest.mark.gpu
def test_graphs_captured_on_one_stream_run_side_by_side():
    """Two graphs with partial results, captured on PyTorch's stream for captures, replayed on two
    streams at once: each gives the eager result's bits."""
    from bit_weight_only_w4a16_amd import block
    g = torch.Generator().manual_seed(1)
    page, d, width = 16, 128, 512
    kc, vc = (torch.randn(2 * width, 2, page, d, generator=g).half().cuda() for _ in range(2))
    table = torch.randperm(2 * width, generator=g).to(torch.int32).view(2, width).cuda()
    ctx = torch.tensor([8000, 7000], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    assert block.awq_attn_tree_workspace_bytes(8, 2, width, page, 4, 8, 2, d) > 0
    w = (torch.randn(264, 1024, generator=g) * 0.05).half().cuda()
    layer = awq.QuantLinear.from_weight(w, torch.randn(32, 1024, generator=g).half().cuda())

    def step(q):
        return layer(block.awq_attn_tree(q, kc, vc, table, ctx, cu, 4).view(8, 1024), act="gelu")

    qs = [torch.randn(8, 8, d, generator=g).half().cuda() for _ in range(2)]
    want = [step(q) for q in qs]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in qs]
    for q in qs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(q))
        graphs.append(graph)
    for _ in range(5):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for out, x in zip(outs, want):
            assert torch.equal(out, x)
        for q, x in zip(qs, want):
            assert torch.equal(step(q), x)


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
