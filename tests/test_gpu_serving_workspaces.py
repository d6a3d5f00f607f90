"""GPU checks of the memory that the norm's, cache's and attention's own workspaces take."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import int8_mixed_precision_rowwise_b200 as m
    return m


def held(f):
    """Bytes that are allocated after f() and were not before."""
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    f()
    torch.cuda.synchronize()
    return torch.cuda.memory_allocated() - before


def test_only_attention_takes_the_large_workspace(lib):
    """On a stream without it: the norm's and the cache's calls take less than 1 MB, and so do graphs of them."""
    s = torch.cuda.Stream()
    large = lib.kv_attention_workspace_size(1, 1, 128)
    x, w = torch.ones((4, 512), dtype=torch.float16, device="cuda"), torch.ones(512, dtype=torch.float16, device="cuda")
    cache = lib.Int8KVCache.empty(4, 1, 16, 64)
    K = torch.ones((2, 1, 64), dtype=torch.float16, device="cuda")
    table, n, at = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([[0, 1, 2]], [2], [0, 2]))
    keys = lambda: [k for d in (lib._serving_workspaces, lib._captured_workspaces) for k in d if k[1] == s.cuda_stream]
    for d in (lib._serving_workspaces, lib._captured_workspaces):  # torch hands out a stream more than once
        for k in [k for k in d if k[1] == s.cuda_stream]:
            del d[k]

    def small():
        with torch.cuda.stream(s):
            lib.add_rmsnorm_quantize(x, w, threshold=0.5)
            cache.append(K, K, table, n, at)
            cache.read(table, n, at, 2)

    assert 0 < held(small) < 1 << 20 and held(small) == 0
    graph = torch.cuda.CUDAGraph()

    def capture():
        with torch.cuda.graph(graph, stream=s):
            lib.add_rmsnorm_quantize(x, w, threshold=0.5)
            cache.append(K, K, table, n, at)

    assert 0 < held(capture) < 1 << 20 and len(keys()) == 2
    small()
    assert len(keys()) == 1  # the graph's is the graph's alone now
    graph.replay()

    def attend():
        with torch.cuda.stream(s):
            cache.attend(K, table, n, at)

    assert large <= held(attend) < large + (1 << 20)
    assert all(lib.read_status(ws, clear=False) == 0 for ws in lib.workspaces(0))


def test_a_graph_keeps_its_workspace_when_the_stream_goes_on(lib):
    """Replays after the binding has let go of the graph's workspaces, with other allocations and captures since."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((40, 4096), generator=g, device="cuda").half()
    w = torch.ones(4096, dtype=torch.float16, device="cuda")
    cache = lib.Int8KVCache.empty(80, 2, 16, 128)
    K = torch.randn((1200, 2, 128), generator=g, device="cuda").half()
    table, n, at = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([list(range(80))], [1200], [0, 1200]))
    cache.append(K, K, table, n, at)
    Q = torch.randn((1, 8, 128), generator=g, device="cuda").half()
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    want = lib.add_rmsnorm_quantize(x, w, threshold=3.0)[:3], cache.attend(Q, table, n, one, max_new=1)
    s = torch.cuda.Stream()
    graphs = []
    for _ in range(3):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = lib.add_rmsnorm_quantize(x, w, threshold=3.0)[:3], cache.attend(Q, table, n, one, max_new=1)
        graphs.append((graph, got))
        with torch.cuda.stream(s):
            cache.attend(Q, table, n, one, max_new=1)
            lib.add_rmsnorm_quantize(x, w, threshold=3.0)
    dirt = torch.full((256 << 20,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for graph, (codes, out) in graphs:
            for t in (*codes, out):
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(codes, want[0])) and torch.equal(out, want[1])
    assert bool((dirt == 255).all())
