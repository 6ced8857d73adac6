"""The attention's tiles of 128 query rows one at a time and in pairs, on both sides of the rule that chooses
between them, whole and cut between CTAs, over bf16 pages, over an e4m3 cache that is expanded first and over
e4m3 pages expanded tile by tile: chosen rows against the float64 oracle."""
import numpy as np
import pytest

import gpu_util as G
import kv_rows as R
import kv_util as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _sms():
    import torch
    return torch.cuda.get_device_properties(0).multi_processor_count


def _pairs(T, heads, g):
    """Whether a call of T tokens takes pairs: more pairs (of 2 * (128 // g) tokens) than half of the SMs."""
    return -(-T // (2 * (128 // g))) * heads > _sms() // 2


def _most_single(heads, g):
    """The most tokens that are still dealt as single tiles."""
    return _sms() // 2 // heads * 2 * (128 // g)


def _run(s, rows, what):
    import torch
    from bit_mixture_experts_gb300 import _lib
    out, lse = s.cache.attention(s.q, s.batch, return_lse=True)
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 0
    R.check_rows(s, out, lse, rows, what=what)
    again = s.cache.attention(s.q, s.batch, return_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("over", [0, 1, 37])
@pytest.mark.parametrize("past", [0, 700])
@pytest.mark.parametrize("d,heads,g,page", [(128, 2, 8, 64), (64, 8, 16, 16), (128, 4, 5, 48)])
def test_prompts_on_both_sides_of_the_rule(d, heads, g, page, past, over):
    T = _most_single(heads, g) + over
    assert _pairs(T, heads, g) == (over > 0)
    s = K.Setup([T], [T + past], heads=heads, g=g, d=d, page=page, seed=T + past)
    # rows from the first to the last tile, and the last pair's (which may have one tile alone)
    _run(s, np.union1d(R.spread(0, T, 10), R.spread(max(0, T - 2 * (128 // g)), T, 3)), f"T={T}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,page", [(128, 64), (64, 128)])
def test_pairs_over_a_long_context(d, page, fmt):
    """Pairs against many more key tiles than a share has: every item is cut between CTAs.  The e4m3 cache is
    expanded before."""
    heads, g = 8, 16
    T = _most_single(heads, g) + 5
    assert _pairs(T, heads, g)
    s = K.Setup([T], [T + 9000], heads=heads, g=g, d=d, page=page, seed=d)
    if fmt == "e4m3":
        _quantised(s, d)
        from bit_mixture_experts_gb300 import _lib
        one = s.cache.batch(s.idx[0], s.idx[1], s.idx[2], 1)
        size = _lib.moe_kv_attention_workspace_size
        assert size(s.cache.struct, s.batch.struct, s.hq) > size(s.cache.struct, one.struct, s.hq)
    _run(s, R.spread(0, T, 5), fmt)


def _quantised(s, seed):
    """Gives a bf16 Setup an e4m3 cache of random codes, scales of four sizes, instead."""
    import torch
    from bit_mixture_experts_gb300 import PagedKVCache
    r = np.random.default_rng(seed)
    pools = []
    for _ in range(2):
        codes = r.integers(0, 126, s.cache.k.shape, dtype=np.uint8) | (r.integers(0, 2, s.cache.k.shape, dtype=np.uint8) << 7)
        # values of about 1: codes up to 126 are 448 at most, spread evenly over the logarithm
        scale = np.exp2(r.integers(-9, -5, s.cache.k.shape[:3])).astype(np.float32)
        pools.append((torch.from_numpy(codes).view(torch.float8_e4m3fn).to(s.dev), torch.from_numpy(scale).to(s.dev)))
    s.fmt = "e4m3"
    s.cache = PagedKVCache.from_tensors(pools[0][0], pools[1][0], pools[0][1], pools[1][1])
    s.batch = s.cache.batch(*s.idx, s.T)


@pytest.mark.parametrize("past", [30, 1500])
@pytest.mark.parametrize("d,page", [(128, 64), (64, 16)])
def test_pairs_over_e4m3_pages_expanded_tile_by_tile(d, page, past):
    """Many sequences of fewer than two pairs on average: the e4m3 pages are not expanded before."""
    from bit_mixture_experts_gb300 import _lib
    heads, g, n = 2, 8, 60  # two pairs of 32 tokens each, the second not full
    B = _sms() // (2 * 2 * heads) + 2
    s = K.Setup([n] * B + [1], [n + past + 7 * b for b in range(B)] + [400], heads=heads, g=g, d=d, page=page, seed=past)
    _quantised(s, past)
    assert _pairs(s.T, heads, g) and s.T * g < 4 * 128 * (B + 1)
    one = s.cache.batch(*s.idx, 1)
    size = _lib.moe_kv_attention_workspace_size
    assert size(s.cache.struct, s.batch.struct, s.hq) == size(s.cache.struct, one.struct, s.hq)
    _run(s, np.append(R.spread(0, s.T - 1, 24), s.T - 1), f"past={past}")
