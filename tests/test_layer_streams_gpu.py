"""The layer on several streams and in graphs: no call reads what another's is writing."""
import pytest

import gpu_util as G

pytestmark = pytest.mark.gpu

H, E, K, F = 256, 64, 4, 256
# fused decode; routing in one block and in several, with and without the combine in the down projection
FORMS = [(4, False), (100, False), (600, False), (600, True)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.fixture(scope="module")
def weights():
    return G.workload((600, H, E, K, F, False), 2)


def make(weights, fuse=False, gate=None):
    from bit_mixture_experts_gb300.layer import MoELayerW4
    return MoELayerW4(H, E, K, F, weights, device=G.torch_dev(), impl="auto" if not fuse else "tc", fuse_combine=fuse,
                      gate=gate)


def inputs(T, n):
    """n calls' inputs, each with experts of its own liking."""
    import torch
    gen = torch.Generator().manual_seed(T)
    return [((torch.randn((T, H), generator=gen) * 0.5).bfloat16().to(G.torch_dev()),
             (torch.randn((T, E), generator=gen) + 2 * torch.randn(E, generator=gen)).to(G.torch_dev())) for _ in range(n)]


def no_error():
    import torch

    from bit_mixture_experts_gb300 import _lib
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 0


@pytest.mark.parametrize("T,fuse", FORMS)
def test_the_first_call_is_on_another_stream(weights, T, fuse):
    """While the current stream is busy: what the call takes is made, and zeroed, on its own stream."""
    import torch

    from bit_mixture_experts_gb300 import ExpertGate, ResidualNorm
    (x, logits), = inputs(T, 1)
    want = make(weights, fuse).forward(x, logits)
    norm = ResidualNorm()
    follows = make(weights, fuse, ExpertGate(K)).forward_residual(x, logits, x, norm)
    no_error()
    for as_handle in (False, True):
        layer, gated = make(weights, fuse), make(weights, fuse, ExpertGate(K))
        side = torch.cuda.Stream()
        s = side.cuda_stream if as_handle else side
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        got = layer.forward(x, logits, stream=s)
        r, n = gated.forward_residual(x, logits, x, norm, stream=s)
        side.synchronize()
        assert torch.equal(got.cpu(), want.cpu())
        assert torch.equal(r.cpu(), follows[0].cpu()) and torch.equal(n.cpu(), follows[1].cpu())
        no_error()


@pytest.mark.parametrize("T,fuse", FORMS)
def test_two_streams(weights, T, fuse):
    import torch
    layer, calls = make(weights, fuse), inputs(T, 2)
    want = [layer.forward(*c) for c in calls]
    no_error()
    assert not torch.equal(*want)
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [[torch.empty_like(w) for _ in range(20)] for w in want]
    torch.cuda.synchronize()
    for i in range(20):
        for s, c, o in zip(streams, calls, outs):
            layer.forward(*c, out=o[i], stream=s)
    no_error()
    for w, o in zip(want, outs):
        assert all(torch.equal(x, w) for x in o)
    names = "counts", "perm", "y"
    a, b = (layer.buffers(T, s) for s in streams)
    assert not any(a[n].data_ptr() == b[n].data_ptr() for n in names)


@pytest.mark.parametrize("warm", [True, False])
@pytest.mark.parametrize("T,fuse", FORMS)
def test_graphs_beside_each_other_and_eager_calls(weights, T, fuse, warm):
    """Two graphs of two calls each, captured with and without a call before, replayed on two streams beside calls."""
    import torch
    layer, calls = make(weights, fuse), inputs(T, 5)
    fresh = make(weights, fuse)
    want = [fresh.forward(*c) for c in calls]
    if warm:
        layer.forward(*calls[0])
    no_error()
    graphs, outs = [], []
    for pair in (calls[:2], calls[2:4]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([layer.forward(*c) for c in pair])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    eager = [torch.empty_like(want[4]) for _ in range(10)]
    torch.cuda.synchronize()
    for i in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        layer.forward(*calls[4], out=eager[i])
    no_error()
    for got, w in zip(outs[0] + outs[1] + eager, want[:4] + [want[4]] * 10):
        assert torch.equal(got, w)


def test_relaxed_capture():
    """Memory made and zeroed beside a capture, which goes on; the thread's mode is the old one afterwards."""
    import ctypes

    import torch

    from bit_mixture_experts_gb300 import _lib
    c = torch.full((1001,), 7, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream(priority=-1)  # (captures are on streams of the usual priority)
    mode = ctypes.c_int32(1)
    _lib._call("moe_exchange_capture_mode", ctypes.byref(mode))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with torch.cuda.stream(side), _lib.relaxed_capture():
            b = torch.zeros(50_000_000, dtype=torch.uint8, device="cuda")
            side.synchronize()
        c.add_(1)
    _lib._call("moe_exchange_capture_mode", ctypes.byref(mode))
    assert mode.value == 1
    assert not b.any() and (c == 7).all()
    g.replay()
    torch.cuda.synchronize()
    assert (c == 8).all() and not b.any()


def test_a_chain_on_two_streams_and_in_graphs():
    import torch

    import workloads
    from bit_mixture_experts_gb300.layer import MoEDecodeChain
    shape = workloads.LayerShape(H=H, E=E, k=K, F=128)
    chain = MoEDecodeChain(H, E, K, 128, [workloads.make_weights(shape, seed=l) for l in range(2)],
                           [workloads.router_weight_bits(shape, seed=l) for l in range(2)], device=G.torch_dev(), impl="gemv")
    xs = [x for x, _ in inputs(4, 4)]
    want = [chain.forward(x).clone() for x in xs]
    no_error()
    streams = [torch.cuda.Stream() for _ in xs[:2]]
    outs = [[], []]
    graphs, kept = [], []
    for x in xs[2:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kept.append(chain.forward(x))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(10):
        for x, s, o, g in zip(xs, streams, outs, graphs):
            with torch.cuda.stream(s):
                o.append(chain.forward(x).clone())
                g.replay()
    no_error()
    for w, o in zip(want, outs):
        assert all(torch.equal(x, w) for x in o)
    assert all(torch.equal(x, w) for x, w in zip(kept, want[2:]))


@pytest.mark.parametrize("T,fuse", FORMS)
def test_a_capture_that_pytorch_did_not_begin(weights, T, fuse):
    """Nothing that is allocated later takes the memory that its replays write to."""
    import ctypes

    import torch
    rt = ctypes.CDLL("libcudart.so.13")
    layer, calls = make(weights, fuse), inputs(T, 2)
    fresh = make(weights, fuse)
    want = [fresh.forward(*c) for c in calls]
    no_error()
    x, logits = (t.clone() for t in calls[0])
    out = torch.empty_like(x)
    st = torch.cuda.Stream()
    handle, graph, run = ctypes.c_void_p(st.cuda_stream), ctypes.c_void_p(), ctypes.c_void_p()
    torch.cuda.synchronize()
    assert rt.cudaStreamBeginCapture(handle, 0) == 0
    with torch.cuda.stream(st):
        layer.forward(x, logits, out)
    assert rt.cudaStreamEndCapture(handle, ctypes.byref(graph)) == 0
    assert rt.cudaGraphInstantiate(ctypes.byref(run), graph, ctypes.c_ulonglong(0)) == 0
    with torch.cuda.stream(st):  # what would be handed out again
        others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda")
                  for n in [16, 512, 1024, 4096, 1 << 16, 1 << 18, 1 << 20, T * K * F * 2, T * K * H * 2] * 20]
    for c, w in zip(calls, want):
        x.copy_(c[0])
        logits.copy_(c[1])
        torch.cuda.synchronize()
        assert rt.cudaGraphLaunch(run, handle) == 0
        no_error()
        assert torch.equal(out, w)
    assert all((t == 7).all() for t in others)
    assert rt.cudaGraphExecDestroy(run) == 0 and rt.cudaGraphDestroy(graph) == 0


def test_graphs_of_pytorch_keep_no_buffers(weights):
    """The layer keeps counters alone of a call that torch.cuda.graph captures."""
    import torch
    layer, ((x, logits),) = make(weights), inputs(600, 1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(x, logits)
    assert len(layer._captured) == 1 and torch.is_tensor(layer._captured[0])


def test_a_gates_scratch_in_such_a_capture():
    import ctypes

    import torch

    from bit_mixture_experts_gb300 import ExpertGate
    rt = ctypes.CDLL("libcudart.so.13")
    gate = ExpertGate(K)
    logits = torch.randn((900, E), device="cuda")
    want = gate.route(logits, 64)
    no_error()
    st = torch.cuda.Stream()
    handle, graph, run = ctypes.c_void_p(st.cuda_stream), ctypes.c_void_p(), ctypes.c_void_p()
    torch.cuda.synchronize()
    assert rt.cudaStreamBeginCapture(handle, 0) == 0
    got = gate.route(logits, 64, stream=st)
    assert rt.cudaStreamEndCapture(handle, ctypes.byref(graph)) == 0
    assert rt.cudaGraphInstantiate(ctypes.byref(run), graph, ctypes.c_ulonglong(0)) == 0
    with torch.cuda.stream(st):
        others = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in [512, 4096, 1 << 14, 1 << 16] * 50]
    torch.cuda.synchronize()
    for _ in range(3):
        assert rt.cudaGraphLaunch(run, handle) == 0
    no_error()
    assert all(torch.equal(a, b) for a, b in zip(got[:6], want[:6]))
    assert all((t == 7).all() for t in others)
    assert rt.cudaGraphExecDestroy(run) == 0 and rt.cudaGraphDestroy(graph) == 0
