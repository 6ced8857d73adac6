"""The paged cache's attention in CUDA graphs: what later calls and other graphs do leaves a graph's scratch
alone, and a graph's replays leave everybody else's memory alone."""
import pytest

import gpu_util as G
import kv_util as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _captured(s, stream=None):
    import torch
    s.cache.attention(s.q, s.batch)  # the first call of a process is not made in a capture
    out = torch.empty((s.T, s.hq, s.d), dtype=torch.bfloat16, device=s.dev)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        s.cache.attention(s.q, s.batch, out=out)
    return graph, out


def test_a_larger_call_after_the_capture():
    """A decode step captured on a stream, then on the same stream a prompt that needs far more scratch, then
    other tensors of all sizes: replays give the step's result and change nothing else."""
    import torch
    from bit_mixture_experts_gb300 import _lib
    # long enough that items are cut: parts go through the scratch
    s = K.Setup([1, 1], [3000, 2000], heads=2, g=8, d=128, page=64, fmt="e4m3", seed=1)
    big = K.Setup([900, 1], [1100, 40], heads=2, g=8, d=128, page=64, fmt="e4m3", seed=2)
    big.cache._workspaces = s.cache._workspaces  # as if both batches were of one cache
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        want = s.cache.attention(s.q, s.batch).clone()
        graph, out = _captured(s, st)
        big.cache.attention(big.q, big.batch)
        torch.cuda.synchronize()
        # whatever memory the larger call gave back is somebody else's now
        others = [torch.full((n << 20,), 0x5a, dtype=torch.uint8, device=s.dev) for n in (64, 32, 32, 16, 8, 4, 2, 1)]
        for _ in range(3):
            out.zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all((t == 0x5a).all() for t in others)
    assert _lib.moe_get_device_error() == 0


def test_two_graphs_replayed_at_once():
    """Graphs captured one after the other on the same stream, replayed on two streams at the same time."""
    import torch
    from bit_mixture_experts_gb300 import _lib
    a = K.Setup([1, 1], [3000, 2000], heads=2, g=8, d=128, page=64, seed=3)
    b = K.Setup([6, 1], [1500, 4000], heads=2, g=8, d=128, page=64, seed=4)
    b.cache._workspaces = a.cache._workspaces
    want = [s.cache.attention(s.q, s.batch) for s in (a, b)]
    graphs = [_captured(s) for s in (a, b)]
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(50):
        for _, out in graphs:
            out.zero_()
        torch.cuda.synchronize()
        for (graph, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            assert torch.equal(out, w)
    assert _lib.moe_get_device_error() == 0
