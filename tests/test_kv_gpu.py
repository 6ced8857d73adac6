"""The paged key/value cache on the GPU (kv.PagedKVCache: append, read, attention) against the float64 oracle
(oracle/kv_ref.py).  Quantised contents are compared bit for bit; attention outputs within the bound that
follows from their roundings (tests/kv_util.py).  Every cache row that no token owns holds NaN."""
import numpy as np
import pytest

from oracle import kv_ref

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


def _new_rows(s, seed, sigma=1.0):
    """New k, v as slices of one fused tensor: [T, heads, d] with padding between the heads and the tokens."""
    import torch
    r = np.random.default_rng(seed)
    x = r.standard_normal((s.T, 2 * s.heads + 3, s.d + 8)) * sigma * np.exp2(r.integers(-20, 20, (s.T, 1, 1)))
    t = torch.from_numpy(x.astype(np.float32)).bfloat16().to(s.dev)
    return t[:, 1:1 + s.heads, :s.d], t[:, 2 + s.heads:2 + 2 * s.heads, :s.d]


BATCHES = [
    ([1], [1]),                                   # the first token of a sequence
    ([5], [3]),                                   # more new tokens than positions: two exist in no page
    ([0, 3, 1, 0], [7, 20, 16, 0]),               # sequences without new tokens, one without any
    ([33, 1, 64, 2], [33, 100, 80, 17]),          # pages that end inside the new tokens
]


@pytest.mark.parametrize("q_lens,kv_lens", BATCHES)
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,heads,page", [(128, 2, 16), (64, 3, 48)])
def test_append_writes_its_slots_alone_and_reads_back(q_lens, kv_lens, fmt, d, heads, page):
    import torch
    s = K.Setup(q_lens, kv_lens, heads=heads, d=d, page=page, fmt=fmt, seed=len(q_lens))
    k, v = _new_rows(s, 1)
    want = []
    for pool, scale, new in ((s.cache.k, s.cache.k_scale, k), (s.cache.v, s.cache.v_scale, v)):
        bits = pool.view(torch.uint8 if fmt == "e4m3" else torch.int16).cpu().numpy().copy()
        sc = None if scale is None else scale.view(torch.int32).cpu().numpy().copy()
        x = new.double().cpu().numpy()
        if fmt == "e4m3":
            codes, s2 = kv_ref.quantise(x)
            s2 = s2.astype(np.float32).view(np.int32)
        else:
            codes = new.contiguous().view(torch.int16).cpu().numpy()
        for b, (n, c) in enumerate(zip(q_lens, kv_lens)):
            for i, p in enumerate(kv_ref.positions(n, c)):
                if p >= 0:
                    page_id, row, t = s.table[b, p // page], p % page, s.cu[b] + i
                    bits[page_id, :, row] = codes[t]
                    if sc is not None:
                        sc[page_id, :, row] = s2[t]
        want.append((bits, sc))
    s.cache.append(k, v, s.batch)
    got = s.cache.read(s.batch)
    _ok()
    vals = s.values()
    for i, (pool, scale) in enumerate(((s.cache.k, s.cache.k_scale), (s.cache.v, s.cache.v_scale))):
        bits, sc = want[i]
        assert np.array_equal(pool.view(torch.uint8 if fmt == "e4m3" else torch.int16).cpu().numpy(), bits)
        if sc is not None:
            assert np.array_equal(scale.view(torch.int32).cpu().numpy(), sc)
        ref = np.zeros((s.T, heads, d))
        for b, (n, c) in enumerate(zip(q_lens, kv_lens)):
            for j, p in enumerate(kv_ref.positions(n, c)):
                if p >= 0:
                    ref[s.cu[b] + j] = vals[i][s.table[b, p // page], :, p % page]
        assert np.array_equal(got[i].double().cpu().numpy(), ref)


def test_append_e4m3_edges():
    """Rows at the scale's steps, ties, zeros, bf16's largest and smallest values, and rows with Inf or NaN."""
    import torch
    d = 64
    rows = []
    for top in (448.0, 449.9, 450.0, 224.0, 1.0, 2.0 ** -126, 2.0 ** -133, 2.0 ** -120, 3.3895314e38, 1.0e-30):
        r = np.linspace(-top, top, d)
        r[0], r[1], r[2], r[3] = top, -top, 0.0, -0.0
        rows.append(r)
    ties = np.array([17.0, 18.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 5 * 2.0 ** -10] * 8)
    ties[-1] = 256.0
    rows += [ties, np.zeros(d), -np.zeros(d)]
    for bad in (np.inf, -np.inf, np.nan):
        r = np.ones(d)
        r[17] = bad
        rows.append(r)
    T = len(rows)
    s = K.Setup([T], [T], heads=1, d=d, page=16, fmt="e4m3")
    x = torch.from_numpy(np.stack(rows)[:, None].astype(np.float32)).bfloat16().to(s.dev)
    s.cache.append(x, -x, s.batch)
    k, v = s.cache.read(s.batch)
    _ok()
    xs = x.double().cpu().numpy()
    codes, sc = kv_ref.quantise(xs[:T - 3])
    ref = kv_ref.TABLE[codes] * sc[..., None]
    with np.errstate(over="ignore"):
        ref = torch.from_numpy(ref.astype(np.float32)).bfloat16().double().numpy()  # 2^128 and below 2^-133
    for got, sign in ((k, 1), (v, -1)):
        g = got.double().cpu().numpy()
        assert np.array_equal(g[:T - 3], sign * ref)
        assert np.isnan(g[T - 3:]).all()


CASES = [  # q_lens, kv_lens, heads, g, d, page
    ([1], [1], 1, 1, 128, 16),
    ([1], [129], 2, 8, 128, 64),
    ([1, 1, 1], [700, 1, 128], 2, 4, 64, 32),
    ([1] * 9, [5, 300, 1000, 64, 127, 128, 129, 2, 640], 2, 8, 128, 16),
    ([2, 7, 0, 1], [2, 300, 50, 400], 1, 5, 128, 48),
    ([16, 3], [270, 1029], 2, 16, 64, 128),
    ([130], [130], 2, 1, 128, 64),
    ([37, 64, 5], [37, 200, 261], 2, 8, 128, 16),
    ([300], [555], 1, 7, 64, 1024),
    ([200, 1], [150, 0], 2, 3, 128, 32),          # rows that see no key: 50 of the first, all of the second
    ([3, 2], [600, 257], 1, 128, 128, 16),
    ([257], [2000], 1, 8, 128, 16),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens,kv_lens,heads,g,d,page", CASES)
def test_attention(q_lens, kv_lens, heads, g, d, page, fmt):
    s = K.Setup(q_lens, kv_lens, heads=heads, g=g, d=d, page=page, fmt=fmt, seed=sum(kv_lens))
    out, lse = s.cache.attention(s.q, s.batch, return_lse=True)
    _ok()
    K.check(s, out, lse, what=f"{q_lens} over {kv_lens} g={g} d={d} page={page} {fmt}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,page", [(128, 32), (64, 16)])
@pytest.mark.parametrize("kind", ["decode", "decode short", "mixed"])
def test_attention_many_sequences(kind, d, page, fmt):
    """More sequences than a warp has lanes and many items per CTA, of one token or of all sizes in turn: what
    one item leaves behind in the CTA must not reach the next.  Several runs, since it would be a matter of time."""
    import torch
    r = np.random.default_rng(d + len(kind))
    if kind == "decode":
        q, kv, heads, g = [1] * 40, r.integers(1, 3000, 40).tolist(), 4, 2
    elif kind == "decode short":
        q, kv, heads, g = [1] * 150, r.integers(1, 300, 150).tolist(), 8, 1
    else:
        q = r.choice([0, 1, 1, 2, 5, 8, 9, 17, 40, 130], 60).tolist()
        kv, heads, g = [int(n + r.integers(0, 400)) for n in q], 4, 4
    s = K.Setup(q, kv, heads=heads, g=g, d=d, page=page, fmt=fmt, seed=31)
    out, lse = s.cache.attention(s.q, s.batch, return_lse=True)
    _ok()
    K.check(s, out, lse, what=kind)
    for _ in range(10):
        again = s.cache.attention(s.q, s.batch, return_lse=True)
    _ok()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale,sigma", [(1.0, 1.0), (0.02, 4.0), (3.0, 2.0)])
def test_attention_scales(scale, sigma, fmt):
    """Flat and nearly one-hot softmax: the running maximum moves a lot or not at all."""
    s = K.Setup([3, 40], [500, 300], heads=1, g=4, d=64, fmt=fmt, sigma=sigma, seed=3)
    out, lse = s.cache.attention(s.q, s.batch, scale=scale, return_lse=True)
    _ok()
    K.check(s, out, lse, scale=scale)


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_attention_running_maximum(order):
    """Scores that rise (every tile moves the maximum, by far) or fall along the sequence."""
    import torch
    n = 1000
    s = K.Setup([2], [n], heads=1, g=2, d=64, page=16, seed=5)
    k = np.zeros((n, 64))
    k[:, 0] = np.arange(n) * (1 if order == "rising" else -1) / 8.0
    kk = s.cache.k.float().cpu().numpy()
    for p in range(n):
        kk[s.table[0, p // 16], 0, p % 16] = k[p]
    s.cache.k.copy_(torch.from_numpy(kk).bfloat16())
    s.q.zero_()
    s.q[..., 0] = 4.0
    out, lse = s.cache.attention(s.q, s.batch, return_lse=True)
    _ok()
    K.check(s, out, lse)


@pytest.mark.parametrize("heads,g,d,page,new,past", [(2, 8, 128, 64, 1, 3000), (1, 5, 64, 16, 6, 999),
                                                     (2, 4, 128, 48, 300, 500)])
def test_attention_e4m3_equals_bf16_of_the_same_values(heads, g, d, page, new, past):
    """A quantised cache and a bf16 cache that holds the values it stands for give the same bits."""
    import torch
    from bit_mixture_experts_gb300 import PagedKVCache
    s = K.Setup([new, new], [new + past, new + past // 3], heads=heads, g=g, d=d, page=page, fmt="e4m3", seed=7)
    a = s.cache.attention(s.q, s.batch, return_lse=True)
    wide = [(x.float() * sc[..., None]).bfloat16() for x, sc in ((s.cache.k, s.cache.k_scale),
                                                                 (s.cache.v, s.cache.v_scale))]
    c2 = PagedKVCache.from_tensors(*wide)
    b = c2.attention(s.q, c2.batch(*s.idx, s.T), return_lse=True)
    _ok()
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("g,new", [(8, 5), (4, 200)])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_ignores_what_later_positions_hold(fmt, g, new):
    """Infinities and NaN in a later token's key or value leave the earlier tokens' results alone."""
    import torch
    s = K.Setup([new, 1], [new + 100, 40], heads=1, g=g, d=128, page=16, fmt=fmt, seed=9)
    clean = s.cache.attention(s.q, s.batch, return_lse=True)
    first = new // 2  # the first bad token
    for i in range(first, new):
        p = 100 + i
        at = s.table[0, p // 16], 0, p % 16
        for pool, scale in ((s.cache.k, s.cache.k_scale), (s.cache.v, s.cache.v_scale)):
            if scale is not None:
                scale[at] = float("nan")
            else:
                pool[at] = (float("nan"), float("inf"), -float("inf"))[i % 3]
    got = s.cache.attention(s.q, s.batch, return_lse=True)
    _ok()
    keep = list(range(first)) + [new]
    for x, y in zip(got, clean):
        assert torch.equal(x[keep], y[keep])
    assert not torch.isfinite(got[0][first:new].float()).any()


def test_attention_strides_scale_and_out():
    import torch
    s = K.Setup([4, 9], [100, 40], heads=2, g=3, d=64, page=32, seed=11)
    wide = torch.zeros((s.hq, s.T, s.d + 16), dtype=torch.bfloat16, device=s.dev)  # heads first, padded rows
    q = wide.transpose(0, 1)[..., 8:8 + s.d]
    q.copy_(s.q)
    out = torch.full((s.T, s.hq, s.d), 7.0, dtype=torch.bfloat16, device=s.dev)
    got = s.cache.attention(q, s.batch, scale=0.3, out=out)
    assert got is out
    _ok()
    K.check(s, out, scale=0.3)


def test_attention_on_another_stream_and_in_a_graph():
    import torch
    s = K.Setup([1, 70], [300, 900], heads=2, g=8, seed=13)
    ref = s.cache.attention(s.q, s.batch)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = s.cache.attention(s.q, s.batch, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    _ok()
    assert torch.equal(ref, got)
    out = torch.zeros_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.cache.attention(s.q, s.batch, out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        _ok()
        assert torch.equal(ref, out)


def test_same_call_same_bits():
    """No sum's order depends on timing."""
    import torch
    s = K.Setup([1, 3, 150], [5000, 2000, 700], heads=2, g=8, seed=15)
    a = s.cache.attention(s.q, s.batch, return_lse=True)
    for _ in range(5):
        b = s.cache.attention(s.q, s.batch, return_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    _ok()


def test_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements, the sequence's pages at its end."""
    import torch
    from bit_mixture_experts_gb300 import PagedKVCache
    small = K.Setup([5], [333], heads=2, g=4, d=128, page=64, seed=17)
    n = (1 << 31) // (2 * 64 * 128) + 64
    cache = PagedKVCache(n, 64, 2, 128)
    off = n - small.cache.num_pages
    for big, sm in ((cache.k, small.cache.k), (cache.v, small.cache.v)):
        big[off:] = sm
    table = torch.where(small.idx[0] >= 0, small.idx[0] + off, small.idx[0])
    batch = cache.batch(table, small.idx[1], small.idx[2], small.T)
    out = cache.attention(small.q, batch)
    k, v = cache.read(batch)
    k2, v2 = small.cache.read(small.batch)
    cache.append(k2 * 2, v2 * 2, batch)
    k3, v3 = cache.read(batch)
    _ok()
    K.check(small, out)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    assert torch.equal(k3, k2 * 2) and torch.equal(v3, v2 * 2)
    del cache
    torch.cuda.empty_cache()


def test_no_tokens_is_no_work():
    import torch
    s = K.Setup([0, 0], [5, 0], heads=1, g=2, d=64, seed=19)
    e = torch.empty((0, 1, 64), dtype=torch.bfloat16, device=s.dev)
    s.cache.append(e, e, s.batch)
    assert s.cache.read(s.batch)[0].shape == (0, 1, 64)
    assert s.cache.attention(s.q, s.batch).shape == (0, 2, 64)
    _ok()


def test_rows_of_no_sequence_are_left_alone():
    import torch
    s = K.Setup([2, 3], [20, 30], heads=1, g=2, d=64, seed=21)
    cu = s.idx[1] + 2  # rows 2..6 of 9 are the sequences'
    batch = s.cache.batch(s.idx[0], cu, s.idx[2], 9)
    q = torch.zeros((9, 2, 64), dtype=torch.bfloat16, device=s.dev)
    q[2:7] = s.q
    out = torch.full_like(q, 7.0)
    s.cache.attention(q, batch, out=out)
    k = torch.full((9, 1, 64), 7.0, dtype=torch.bfloat16, device=s.dev)
    v = k.clone()
    s.cache.read(batch, out=(k, v))
    _ok()
    K.check(s, out[2:7])
    for t in (out, k, v):
        assert (t[:2] == 7).all() and (t[7:] == 7).all()


def test_bad_device_data_is_reported_and_not_followed():
    """Page ids out of the pool, lengths beyond the table, row offsets that decrease: the device error word
    says so, the call ends, and calls on sound data are right afterwards."""
    import torch
    from bit_mixture_experts_gb300 import _lib
    s = K.Setup([2, 140], [100, 300], heads=1, g=4, d=128, seed=23)
    good = s.cache.attention(s.q, s.batch)
    _ok()
    k, v = _new_rows(s, 3)
    table, cu, kv = s.idx
    for page in (-5, s.cache.num_pages, 2 ** 31 - 1):
        t = table.clone()
        t[1, 2] = page
        t[1, 17] = page  # a page of the new tokens too
        b = s.cache.batch(t, cu, kv, s.T)
        for call in (lambda: s.cache.attention(s.q, b), lambda: s.cache.read(b),):
            call()
            assert _lib.moe_get_device_error() == 2
    for bad_kv in (-1, 10 ** 9):
        n = kv.clone()
        n[0] = bad_kv
        s.cache.attention(s.q, s.cache.batch(table, cu, n, s.T))
        assert _lib.moe_get_device_error() == 2
    for bad_cu in ([0, -3, 142], [0, 2, 10 ** 6], [0, 200, 142]):
        c = torch.tensor(bad_cu, dtype=torch.int32, device=s.dev)
        s.cache.attention(s.q, s.cache.batch(table, c, kv, s.T))
        assert _lib.moe_get_device_error() == 2
    before = s.cache.k.clone()
    t = table.clone()
    t[:] = -1
    s.cache.append(k, v, s.cache.batch(t, cu, kv, s.T))
    assert _lib.moe_get_device_error() == 2
    assert torch.equal(before.view(torch.int16), s.cache.k.view(torch.int16))
    again = s.cache.attention(s.q, s.batch)
    _ok()
    assert torch.equal(good, again)


def test_refusals():
    import torch
    from bit_mixture_experts_gb300 import PagedKVCache, _lib
    s = K.Setup([2], [20], heads=2, g=2, d=64, fmt="e4m3")
    c, b = s.cache, s.batch
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device=s.dev)
    for bad in (k.float(), k[:1], k[:, :1], k[..., :32], k.cpu(), k.transpose(1, 2)):
        with pytest.raises(ValueError):
            c.append(bad, k, b)
        with pytest.raises(ValueError):
            c.append(k, bad, b)
    with pytest.raises(ValueError):
        c.read(b, out=(k, k[..., :32]))
    with pytest.raises(ValueError):
        c.attention(s.q.float(), b)
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(_lib.MoeError) as ex:
            c.attention(s.q, b, scale=bad)
        assert ex.value.code == -3
    with pytest.raises(_lib.MoeError) as ex:
        c.attention(s.q[:, :3].contiguous(), b)  # 3 query heads over 2 KV heads
    assert ex.value.code == -3
    odd = torch.zeros((2, 2, 68), dtype=torch.bfloat16, device=s.dev)[..., :64]  # rows not on 16 bytes
    with pytest.raises(_lib.MoeError) as ex:
        c.append(odd, k, b)
    assert ex.value.code == -3
    off = torch.zeros(2 * 2 * 64 + 1, dtype=torch.bfloat16, device=s.dev)[1:].view(2, 2, 64)
    with pytest.raises(_lib.MoeError) as ex:
        c.append(k, off, b)
    assert ex.value.code == -2
    with pytest.raises(ValueError):
        c.batch(s.idx[0].long(), s.idx[1], s.idx[2], 2)
    with pytest.raises(ValueError):
        c.batch(s.idx[0], s.idx[1][:1], s.idx[2], 2)
    with pytest.raises(ValueError):
        PagedKVCache.from_tensors(c.k, c.v)  # no scales
    with pytest.raises(ValueError):
        PagedKVCache(4, 16, 2, 64, fmt="int8")
    _ok()
