"""Attention over long caches, their sums in many parts, against the float64 oracle: flat scores, where a key tile
that is left out shows in the log-sum-exp, and steep ones, where a few keys anywhere in the cache make the output."""
import numpy as np
import pytest

import gpu_util as G
import kv_rows as R
import kv_util as K
from test_kv_pairs_gpu import _quantised

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


# new tokens, keys, query heads per KV head
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,n,g,d", [(1, 131071, 4, 128), (4, 70001, 4, 64), (6, 40000, 8, 128), (40, 33333, 4, 64)])
def test_long_caches(new, n, g, d, fmt):
    import torch
    from bit_mixture_experts_gb300 import _lib
    s = K.Setup([new], [n], heads=1, g=g, d=d, page=64, seed=new)
    if fmt == "e4m3":
        _quantised(s, new)
    # Additions in a row of a sum over keys: at most 35 per key tile (32 in a thread of the 128-row form, four in
    # the thin one), and fewer than 200 to join warps' and CTAs' parts.
    chain = (lambda k: k / 32 + 200) if new * g <= 32 else (lambda k: k * 35 / 128 + 200)
    for scale in (None, 0.5 if fmt == "bf16" else 0.1):
        out, lse = s.cache.attention(s.q, s.batch, scale=scale, return_lse=True)
        torch.cuda.synchronize()
        assert _lib.moe_get_device_error() == 0
        R.check_rows(s, out, lse, R.spread(0, new, 2), scale=scale, chain=chain, what=f"scale {scale}")


@pytest.mark.parametrize("power", [-90, 80])
@pytest.mark.parametrize("new,g", [(1, 4), (4, 4), (8, 4), (60, 4)])
def test_e4m3_values_of_extreme_scales_equal_bf16_ones(new, g, power):
    """Over the scales that the comment of the form for few rows names, weights times scales lose no bits."""
    import torch
    from bit_mixture_experts_gb300 import PagedKVCache, _lib
    s = K.Setup([new], [1500], heads=2, g=g, d=64, page=32, seed=power + 100)
    _quantised(s, new)
    s.cache.v_scale.mul_(2.0 ** power)
    wide = [(x.float() * sc[..., None]).bfloat16() for x, sc in ((s.cache.k, s.cache.k_scale),
                                                                 (s.cache.v, s.cache.v_scale))]
    a = s.cache.attention(s.q, s.batch)
    c2 = PagedKVCache.from_tensors(*wide)
    b = c2.attention(s.q, c2.batch(*s.idx, s.T))
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 0
    assert torch.isfinite(a).all() and a.any(-1).all()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
