"""The paged cache's calls on streams given as torch streams, as raw handles and as the current stream."""
import pytest

import gpu_util as G
import kv_util as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.mark.parametrize("kind", ["stream", "handle", "default"])
def test_calls_on_a_stream_given_in_any_way(kind):
    import torch
    from bit_mixture_experts_gb300 import _lib
    s = K.Setup([1, 70], [3000, 900], heads=2, g=8, seed=13)
    k, v = s.cache.read(s.batch)
    want = s.cache.attention(s.q, s.batch, return_lse=True)
    st = torch.cuda.Stream() if kind != "default" else torch.cuda.default_stream()
    stream = st if kind == "stream" else st.cuda_stream
    assert kind != "default" or stream == 0
    st.wait_stream(torch.cuda.current_stream())
    s.cache.append(k, v, s.batch, stream=stream)
    back = s.cache.read(s.batch, stream=stream)
    got = s.cache.attention(s.q, s.batch, return_lse=True, stream=stream)
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 0
    for a, b in zip((k, v) + want, back + got):
        assert torch.equal(a, b)
    assert st.cuda_stream in s.cache._workspaces
