"""Which buffers a layer's calls take, without a GPU: a set per number of tokens and stream, made on that stream; a captured
call's own."""
import contextlib

import pytest

torch = pytest.importorskip("torch")


class Side:
    """The layer's own stream."""

    def __init__(self):
        self.waits = 0

    def synchronize(self):
        self.waits += 1


class Device:
    """Stands in for PyTorch's streams: `current`, those that are being captured, and on which one memory was made."""

    def __init__(self, monkeypatch):
        from bit_mixture_experts_gb300 import layer
        self.current, self.capturing, self.made, self.pool = 0, set(), [], True
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.current in self.capturing)
        monkeypatch.setattr(torch.cuda, "stream", self.on)
        monkeypatch.setattr(layer, "_on", lambda stream, device: self.on(stream), raising=False)
        monkeypatch.setattr(layer._lib, "_stream", lambda stream=None: self.current if stream is None else stream)
        monkeypatch.setattr(layer._lib, "relaxed_capture", contextlib.nullcontext, raising=False)
        monkeypatch.setattr(layer, "_in_a_graphs_pool", lambda t: self.pool, raising=False)
        for name in ("empty", "zeros"):
            make = getattr(torch, name)
            monkeypatch.setattr(torch, name, lambda *a, name=name, make=make, **kw: self.note(name, make(*a, **kw)))

    def note(self, name, t):
        self.made.append((name, t.data_ptr(), self.current))
        return t

    @contextlib.contextmanager
    def on(self, stream):
        before, self.current = self.current, stream
        yield
        self.current = before


@pytest.fixture
def layer():
    from bit_mixture_experts_gb300 import _lib, build
    from bit_mixture_experts_gb300.layer import MoELayerW4
    build.build()
    self = MoELayerW4.__new__(MoELayerW4)
    self.H, self.E, self.k, self.F, self.device = 128, 64, 4, 128, torch.device("cpu")
    self.impl, self.block_n, self.fuse_combine, self.gate = _lib.IMPL_AUTO, None, True, None
    self._bufs, self._captured, self._side = {}, [], Side()
    return self


NAMES = ("topk_ids", "topk_w", "counts", "offsets", "perm", "inv_perm", "block_map", "num_blocks", "h", "y")


def pointers(b, T):
    scratch = ("decode_ws" if T <= 8 else "workspace", "combine_ws")  # two that are zero between calls
    return {b[n].data_ptr() for n in NAMES + scratch}


@pytest.mark.parametrize("T", [4, 600])
def test_streams_share_no_buffers(layer, monkeypatch, T):
    dev = Device(monkeypatch)
    a = layer.buffers(T)
    assert layer.buffers(T) is a
    b = layer.buffers(T, 7)
    assert layer.buffers(T, 7) is b and not pointers(a, T) & pointers(b, T)
    # made, and zeroed, in order with the stream's calls
    assert {s for _, p, s in dev.made if p in pointers(a, T)} == {0}
    assert {s for _, p, s in dev.made if p in pointers(b, T)} == {7}
    with dev.on(7):
        assert layer.buffers(T) is b
    assert layer.buffers(T) is a
    for x in (a, b):
        assert not x["workspace"].any() if T > 8 else not x["decode_ws"].any()


@pytest.mark.parametrize("T", [4, 600])
def test_captured_calls_share_no_buffers(layer, monkeypatch, T):
    dev = Device(monkeypatch)
    eager = layer.buffers(T, 7)
    dev.capturing.add(7)
    sets = [layer.buffers(T, 7) for _ in range(2)]
    dev.capturing.clear()
    assert layer.buffers(T, 7) is eager
    for x, y in ((eager, sets[0]), (eager, sets[1]), sets):
        assert not pointers(x, T) & pointers(y, T)
    # no fill becomes part of the graph, and what was zeroed stays the layer's
    assert ("zeros", 7) not in {(n, s) for n, p, s in dev.made if p in pointers(sets[0], T) | pointers(sets[1], T)}
    side = layer._side
    assert [t.data_ptr() for t in layer._captured] == [p for n, p, s in dev.made if s is side]
    assert side.waits == 4 == len(layer._captured) and not any(t.any() for t in layer._captured)
    # a capture of the very stream that fills: in the graph then
    dev.capturing.add(side)
    layer.buffers(T, side)
    assert len(layer._captured) == 4
    # a capture that PyTorch keeps no memory for: the layer does
    dev.pool = False
    dev.capturing.add(7)
    b = layer.buffers(T, 7)
    assert any(x is b for x in layer._captured)


def test_a_chains_streams_and_captures_share_no_buffers(monkeypatch):
    from bit_mixture_experts_gb300.layer import MoEDecodeChain
    dev = Device(monkeypatch)
    chain = MoEDecodeChain.__new__(MoEDecodeChain)
    chain.H, chain.E, chain.k, chain.device, chain.layers, chain._bufs = 128, 64, 4, torch.device("cpu"), [None] * 2, {}
    sets = [chain.buffers(4), chain.buffers(4, 7)]
    assert chain.buffers(4) is sets[0] and chain.buffers(4, 7) is sets[1]
    dev.capturing.add(7)
    sets += [chain.buffers(4, 7), chain.buffers(4, 7)]
    dev.capturing.clear()
    assert chain.buffers(4, 7) is sets[1]
    at = [{t.data_ptr() for ts in b.values() for t in ts} for b in sets]
    assert len(set.union(*at)) == sum(len(a) for a in at) == 4 * 10
    for a, s in zip(at, (0, 7, 7, 7)):
        assert {stream for _, p, stream in dev.made if p in a} == {s}
