"""The paged cache's attention where a call could go wrong quietly: values that are not finite under weights
that round to zero, an e4m3 cache that is expanded before the attention, scratch that is too small, forms
chosen by size meeting in one call, and waits that run out (MOE_DEV_TIMEOUT in the device error word, no hang,
sound results once the limit is back)."""
import numpy as np
import pytest

import gpu_util as G
import kv_util as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _ok():
    import torch
    from bit_mixture_experts_gb300 import _lib
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 2, 40, 300])
def test_value_that_is_not_finite_under_a_zero_weight(fmt, d, new):
    """0 x NaN is NaN: a visible key whose weight underflows still passes its NaN on, in every form; a hidden
    one does not."""
    import torch
    s = K.Setup([new], [700], heads=1, g=4, d=d, page=16, fmt=fmt, seed=4)
    s.q.fill_(1.0)
    at = lambda p: (int(s.table[0, p // 16]), 0, p % 16)
    seen, hidden = 5, 699  # the last position: only the last token sees it
    for p in (seen, hidden):
        # scores of at most -448 sqrt(d) < -3500: exp underflows in FP32 beside scores of size 30
        if fmt == "bf16":
            s.cache.k[at(p)] = -448.0
        else:
            s.cache.k[at(p)] = torch.full((d,), -448.0, device=s.dev).to(torch.float8_e4m3fn)
            s.cache.k_scale[at(p)] = 1.0

    def poison(p):
        if fmt == "bf16":
            s.cache.v[at(p)] = float("nan")
        else:
            s.cache.v_scale[at(p)] = float("nan")

    poison(hidden)
    out = s.cache.attention(s.q, s.batch)
    _ok()
    assert torch.isnan(out[-1]).all() and torch.isfinite(out[:-1]).all()
    poison(seen)
    out = s.cache.attention(s.q, s.batch)
    _ok()
    assert torch.isnan(out).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,g", [(8, 4), (4, 8), (3, 8), (5, 5)])
def test_value_that_is_not_finite_and_only_some_rows_see(fmt, new, g):
    """More than 16 query rows: two warps have the same keys, for different rows, and both must notice a value
    that is not finite whichever comes first.  Many calls, since it is a matter of time."""
    import torch
    s = K.Setup([new], [700], heads=2, g=g, d=128, page=16, fmt=fmt, seed=9)
    for p in range(700 - new + 1, 700):  # position p: seen by the new tokens from p on
        at = (int(s.table[0, p // 16]), slice(None), p % 16)
        if fmt == "bf16":
            s.cache.v[at] = float("nan")
        else:
            s.cache.v_scale[at] = float("nan")
    outs = [s.cache.attention(s.q, s.batch) for _ in range(200)]
    _ok()
    for out in outs:
        assert torch.isfinite(out[0]).all() and torch.isnan(out[1:]).all()


@pytest.mark.parametrize("q_lens,kv_lens,g,d,page", [([700], [900], 2, 128, 16), ([600, 1, 580], [600, 1, 1100], 4, 64, 48),
                                                     ([300, 299, 0], [300, 200, 70], 8, 128, 64)])
def test_many_rows_over_an_e4m3_cache(q_lens, kv_lens, g, d, page):
    """Many query rows per sequence: the cache is expanded to bf16 in the workspace first."""
    import torch
    from bit_mixture_experts_gb300 import _lib
    s = K.Setup(q_lens, kv_lens, heads=2, g=g, d=d, page=page, fmt="e4m3", seed=6)
    wide = K.Setup([1] * len(q_lens), kv_lens, heads=2, g=g, d=d, page=page, fmt="e4m3", seed=6)
    # (the workspace shows it: the parts of cut items alone otherwise)
    size = _lib.moe_kv_attention_workspace_size
    assert size(s.cache.struct, s.batch.struct, s.hq) > size(wide.cache.struct, wide.batch.struct, s.hq)
    out, lse = s.cache.attention(s.q, s.batch, return_lse=True)
    _ok()
    K.check(s, out, lse)
    # a page that does not exist is reported, not followed, and its sequence alone is wrong
    t = s.idx[0].clone()
    t[0, 3] = s.cache.num_pages
    bad = s.cache.attention(s.q, s.cache.batch(t, *s.idx[1:], s.T))
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 2
    assert torch.equal(bad[s.cu[1]:], out[s.cu[1]:])
    again = s.cache.attention(s.q, s.batch)
    _ok()
    assert torch.equal(again, out)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,heads,g", [(1, 2, 4), (90, 2, 4), (2600, 2, 8), (700, 4, 4)])
def test_scratch_too_small_is_refused(fmt, new, heads, g):
    import torch
    from bit_mixture_experts_gb300 import _lib
    s = K.Setup([new], [new + 40], heads=heads, g=g, d=64, fmt=fmt, seed=8)
    need = _lib.moe_kv_attention_workspace_size(s.cache.struct, s.batch.struct, s.hq)
    ws = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device=s.dev)
    with pytest.raises(_lib.MoeError) as ex:
        s.cache.attention(s.q, s.batch, workspace=ws[:need - 16])
    assert ex.value.code == -4
    out = s.cache.attention(s.q, s.batch, workspace=ws[:need])
    _ok()
    assert (ws[need:] == 0x5a).all()  # and no more than it asks for is written
    assert torch.equal(out, s.cache.attention(s.q, s.batch))


@pytest.mark.parametrize("T,past", [(255, 700), (1200, 0), (1201, 300), (2470, 100)])
def test_either_side_of_the_rule_for_tiles(T, past):
    """Single query tiles and pairs, cut and whole items: T tokens of one sequence, some rows checked."""
    import torch
    s = K.Setup([T], [T + past], heads=2, g=8, d=64, page=64, seed=T)
    out, lse = s.cache.attention(s.q, s.batch, return_lse=True)
    _ok()
    # the same tokens one small batch at a time take other forms: every row within the bound of both
    rows = np.unique(np.concatenate([np.arange(0, T, max(1, T // 12)), [T - 1]]))
    for i in rows:
        n = torch.tensor([past + i + 1], dtype=torch.int32, device=s.dev)
        cu = torch.tensor([0, 1], dtype=torch.int32, device=s.dev)
        b = s.cache.batch(s.idx[0], cu, n, 1)
        one, one_lse = s.cache.attention(s.q[i:i + 1].contiguous(), b, return_lse=True)
        # twice the bound of tests/kv_util.py, with |v| <= 5.5 (the largest of these normal values): weights and
        # output rounded to bf16 on both sides
        tol = 2 * (2.0 ** -8 * one.float().abs() + 2.0 ** -8 * 5.5 + 2.0 ** -12)
        assert ((one.float() - out[i:i + 1].float()).abs() <= tol).all()
        assert ((one_lse - lse[i:i + 1]).abs() <= 1e-4).all()
    _ok()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens,kv_lens", [([1] * 8, [3000] * 8), ([700], [1500]), ([40] * 4 + [1] * 4, [2000] * 8)])
def test_waits_that_run_out(fmt, q_lens, kv_lens):
    import torch
    from bit_mixture_experts_gb300 import _lib
    s = K.Setup(q_lens, kv_lens, heads=2, g=8, d=128, page=64, fmt=fmt, seed=12)
    good = s.cache.attention(s.q, s.batch)
    _ok()
    # 0.2 us: a wait on memory that is still open after its first check runs out
    _lib.moe_set_wait_limit_ns(200)
    code = 0
    try:
        for _ in range(20):
            s.cache.attention(s.q, s.batch)
            torch.cuda.synchronize()
            code = _lib.moe_get_device_error()
            if code:
                break
    finally:
        _lib.moe_set_wait_limit_ns(1_000_000_000)
    assert code == 3
    for _ in range(3):
        again = s.cache.attention(s.q, s.batch)
        _ok()
        assert torch.equal(good, again)
