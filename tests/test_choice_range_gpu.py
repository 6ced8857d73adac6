"""Choices from outside that name an expert that does not exist: reported by every form of the layer and of the sort, at
every size around their borders, without an access out of range; the next call is as ever."""
import pytest

import gpu_util as G

pytestmark = pytest.mark.gpu

BAD_INDEX = 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.fixture(scope="module")
def layer():
    from bit_mixture_experts_gb300.layer import MoELayerW4
    d = G.workload((257, 256, 64, 4, 256, False), 3)
    return MoELayerW4(256, 64, 4, 256, d, device=G.torch_dev())


@pytest.mark.parametrize("bad", [64, -1, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("T", [1, 8, 9, 16, 17, 100, 256, 257])
def test_layer(layer, T, bad):
    import torch

    from bit_mixture_experts_gb300 import ResidualNorm, _lib
    gen = torch.Generator().manual_seed(T)
    x = torch.randn((T, 256), generator=gen).bfloat16().cuda()
    ids = torch.randint(0, 64, (T, 4), generator=gen).int().cuda()
    w = torch.rand((T, 4), generator=gen).cuda()
    norm = ResidualNorm()
    want = layer.forward_residual(x, None, x, norm, choice=(ids, w))
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 0
    for at in (0, T * 4 - 1):
        other = ids.clone()
        other.view(-1)[at] = bad
        layer.forward_residual(x, None, x, norm, choice=(other, w))
        torch.cuda.synchronize()
        assert _lib.moe_get_device_error() == BAD_INDEX
        again = layer.forward_residual(x, None, x, norm, choice=(ids, w))
        torch.cuda.synchronize()
        assert _lib.moe_get_device_error() == 0
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("T,E,k", [(1, 5, 1), (128, 64, 8), (129, 64, 8), (1024, 7, 1), (5000, 300, 2)])
def test_sort(T, E, k):
    import torch

    from bit_mixture_experts_gb300 import _lib
    ids = torch.arange(T * k, device="cuda").remainder(E).int().view(T, k)
    ids[T // 2, k - 1] = E
    w = torch.ones((T, k), device="cuda")
    out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in
           ((E,), (E + 1,), (T * k,), (T * k,), (_lib.moe_block_map_capacity(T, E, k, 64), 3), (1,))]
    ws = torch.zeros(max(16, _lib.moe_route_workspace_size(T, E, k, 64)), dtype=torch.uint8, device="cuda")
    for good in (False, True):
        if good:
            ids[T // 2, k - 1] = 0
        _lib.moe_route_gated(None, T, E, k, None, 64, ids, w, *out, ws)
        torch.cuda.synchronize()
        assert _lib.moe_get_device_error() == (0 if good else BAD_INDEX)
        assert int(out[0].sum()) == T * k and (out[2][out[3].long()].cpu() == torch.arange(T * k)).all()
