"""Chosen logits that are further apart than 32 bits hold: an expert forced by +inf or a very large logit among others
masked with the type's lowest value.  The weights are the definition's, that of the largest among them."""
import numpy as np
import pytest

from oracle import gate_ref
from test_gate_gpu import make

pytestmark = pytest.mark.gpu

LOWEST = float(np.finfo(np.float32).min)
# u = 2^-24: e^x off by 4 u, sum and division 2 u, the sum over the chosen 6 u and its additions 5 u, division and scale 2 u
REL = 19 * 2.0 ** -24


def setup_module():
    import gpu_util
    gpu_util.ensure_built()


def far(E):
    """Tokens, a row each."""
    l = np.full((6, E), LOWEST, np.float32)
    l[0, [3, 7]] = np.inf, 1.0
    l[1] = -3e38
    l[1, 5] = 3e38
    l[2, [E - 1, 2]] = np.inf, np.inf
    l[3, 4] = 2e38
    l[4, [1, 6]] = 3e38, -2e38
    l[5, 3] = 0.5  # the usual mask
    return l


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top", [(6, 16, 4, 1, 1), (6, 256, 8, 8, 4), (6, 512, 32, 1, 1), (9000, 256, 8, 8, 4),
                                              (9000, 64, 8, 1, 1)])
def test_gates(T, E, k, groups, top, score, with_bias, renorm):
    import torch

    from bit_mixture_experts_gb300 import _lib
    l = far(E)
    b = np.zeros(E, np.float32) if with_bias else None
    kw = dict(score=score, groups=groups, top_groups=top, group_score="max", renorm=renorm, scale=2.5)
    rows = np.arange(T) % len(l)
    ids, w = make(k, b, **kw).choose(torch.tensor(l[rows], device="cuda"))
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 0
    want_ids, want = gate_ref.choose(l, k, bias=b, **kw)
    assert (want.sum(1) > 1.5).all()  # (each token has one whose score is not small)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids[rows])
    np.testing.assert_allclose(w.double().cpu().numpy(), want[rows], rtol=REL, atol=0)


@pytest.mark.parametrize("T,E,k", [(1, 16, 4), (100, 256, 8), (4096, 256, 8), (300, 1000, 32)])
def test_route(T, E, k):
    """moe_route in one block and in many: finite logits alone, as it takes no others."""
    from test_route_gpu import run_route
    l = np.clip(far(E)[np.arange(T) % 6], LOWEST, -LOWEST)
    got = run_route(l, k, 64)
    ids, w = gate_ref.choose(l[:6], k)
    np.testing.assert_array_equal(got["topk_ids"][:6], ids)
    np.testing.assert_allclose(got["topk_w"].astype(np.float64), w[np.arange(T) % 6], rtol=REL, atol=0)


@pytest.mark.parametrize("T", [1, 6, 40])
def test_layer(T):
    """The layer's own choice, in the fused decode kernel and before the GEMMs."""
    import gpu_util as G
    import torch

    from bit_mixture_experts_gb300 import _lib
    from bit_mixture_experts_gb300.layer import MoELayerW4
    d = G.workload((T, 256, 64, 4, 128, False), 1)
    layer = MoELayerW4(256, 64, 4, 128, d, device=G.torch_dev())
    x, _ = G.to_dev_inputs(d)
    l = np.clip(far(64)[np.arange(T) % 6], LOWEST, -LOWEST)
    out = layer.forward(x, torch.tensor(l, device=x.device))
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 0
    b = layer.buffers(T)
    ids, w = gate_ref.choose(l, 4)
    np.testing.assert_array_equal(b["topk_ids"].cpu().numpy(), ids)
    np.testing.assert_allclose(b["topk_w"].double().cpu().numpy(), w, rtol=REL, atol=0)
    assert torch.isfinite(out).all()
