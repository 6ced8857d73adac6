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
