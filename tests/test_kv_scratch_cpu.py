"""Which scratch the paged cache's attention hands to a call, without a GPU: one per stream that grows, and
one of its own for each call that a graph captures."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def cache(monkeypatch):
    from bit_mixture_experts_gb300 import PagedKVCache, _lib
    monkeypatch.setattr(_lib, "moe_kv_attention_workspace_size", lambda cache, batch, q_heads: batch)
    monkeypatch.setattr(_lib, "_stream", lambda stream=None: 7)
    self = PagedKVCache.__new__(PagedKVCache)
    self.device, self.struct, self._workspaces = torch.device("cpu"), None, {}
    self.capture = lambda on: monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: on)
    self.capture(False)
    return self


def _batch(need):
    return types.SimpleNamespace(workspace={}, struct=need)


def _address(ws):
    return ws[0] if isinstance(ws, tuple) else ws.data_ptr()


def test_a_captured_call_has_scratch_of_its_own(cache):
    small, large = _batch(4096), _batch(1 << 20)
    eager = cache._workspace(small, 4, None)
    cache.capture(True)
    one, two = cache._workspace(small, 4, None), cache._workspace(small, 4, None)
    cache.capture(False)
    # not the stream's, which a larger call replaces and other calls use, and not another capture's
    assert len({_address(w) for w in (eager, one, two)}) == 3
    assert all(isinstance(w, torch.Tensor) and w.nbytes == 4096 for w in (one, two))
    assert cache._workspace(small, 4, None) == eager
    grown = cache._workspace(large, 4, None)
    assert grown[1] == 1 << 20 and cache._workspace(small, 4, None) == grown


def test_a_capture_that_comes_first_leaves_nothing_behind(cache):
    cache.capture(True)
    cache._workspace(_batch(4096), 4, None)
    cache.capture(False)
    assert cache._workspaces == {}
