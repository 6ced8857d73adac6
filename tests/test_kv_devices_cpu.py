"""What the paged cache refuses because a kernel could not reach it, without a GPU: pools in host memory,
calls while another device is the current one, scratch that is no device memory or not what it says."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def launched(monkeypatch):
    """Names of the library's entry points that were called, in place of the calls."""
    from bit_mixture_experts_gb300 import _lib
    calls = []
    monkeypatch.setattr(_lib, "load", lambda *a: None)
    monkeypatch.setattr(_lib, "_call", lambda name, *a: calls.append(name))
    monkeypatch.setattr(_lib, "_stream", lambda stream=None: 7)
    return calls


def _pools():
    return [torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16) for _ in range(2)]


def test_pools_in_host_memory_are_refused(launched):
    from bit_mixture_experts_gb300 import PagedKVCache
    with pytest.raises(ValueError, match="CUDA"):
        PagedKVCache.from_tensors(*_pools())
    with pytest.raises(ValueError, match="CUDA"):
        PagedKVCache(2, 16, 2, 64, device="cpu")


@pytest.fixture
def cache(launched, monkeypatch):
    """A cache that takes host tensors for those of the CUDA device 0, which is the current one."""
    from bit_mixture_experts_gb300 import PagedKVCache
    self = PagedKVCache.__new__(PagedKVCache)
    self.device, self.struct, self._workspaces = torch.device("cpu"), None, {}
    self.k, self.v = _pools()
    self.num_pages, self.heads, self.page_size, self.d = self.k.shape
    monkeypatch.setattr(PagedKVCache, "_workspace", lambda *a: (256, 1 << 20))
    self.device_index = 0
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return self


def _calls(cache, **kw):
    batch = types.SimpleNamespace(T=3, struct=None)
    new = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    return {"append": lambda: cache.append(new, new, batch), "read": lambda: cache.read(batch),
            "attention": lambda: cache.attention(new, batch, **kw)}


@pytest.mark.parametrize("call", ["append", "read", "attention"])
def test_another_device_is_current(cache, launched, monkeypatch, call):
    _calls(cache)[call]()
    assert launched == ["moe_kv_" + call]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        _calls(cache)[call]()
    assert launched == ["moe_kv_" + call]


def test_scratch_of_the_wrong_kind_is_refused(cache, launched):
    ws = torch.zeros(4096, dtype=torch.uint8)
    _calls(cache, workspace=ws)["attention"]()
    assert launched == ["moe_kv_attention"]
    for bad in (ws[::2], ws.to("meta")):
        with pytest.raises(ValueError, match="workspace"):
            _calls(cache, workspace=bad)["attention"]()
    assert launched == ["moe_kv_attention"]
