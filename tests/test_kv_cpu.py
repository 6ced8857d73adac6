"""The paged key/value cache without a GPU: argument checks of the C ABI that fail before any CUDA call, and
the oracle's own pins (e4m3 against torch's conversion, attention against a closed form)."""
import ctypes

import numpy as np
import pytest

from oracle import kv_ref


@pytest.fixture(scope="module")
def lib():
    from bit_mixture_experts_gb300 import _lib, build
    build.build()
    return _lib.load()


def _structs(k=256, sc=256, num_pages=8, page=16, heads=2, d=128, fmt=0, idx=4, B=2, width=4, T=3):
    from bit_mixture_experts_gb300 import _lib
    return (_lib.KVCache(k, k, sc, sc, num_pages, page, heads, d, fmt),
            _lib.KVBatch(idx, idx, idx, B, width, T))


def _append(lib, ptr=256, stride=256, head=128, **kw):
    return lib.moe_kv_append(ptr, stride, head, ptr, stride, head, *_structs(**kw), None)


def _attention(lib, ptr=256, stride=1024, head=128, q_heads=8, scale=0.1, lse=None, out=256, ws=256, ws_bytes=1 << 40,
               **kw):
    return lib.moe_kv_attention(ptr, stride, head, q_heads, scale, *_structs(**kw), out, lse, ws, ws_bytes, None)


BAD = [(dict(d=96), -3), (dict(d=256), -3), (dict(page=8), -3), (dict(page=24), -3), (dict(page=2048), -3),
       (dict(heads=0), -3), (dict(num_pages=0), -3), (dict(num_pages=1 << 27, page=16, heads=1), -3),
       (dict(T=-1), -3), (dict(T=(1 << 20) + 1), -3), (dict(B=0), -3), (dict(B=65537), -3), (dict(width=0), -3),
       (dict(width=1 << 27), -3), (dict(fmt=2), -7), (dict(k=None), -1), (dict(k=264), -2), (dict(idx=None), -1),
       (dict(idx=6), -2), (dict(fmt=1, sc=None), -1), (dict(fmt=1, sc=260), -2), (dict(ptr=None), -1),
       (dict(ptr=264), -2), (dict(stride=257), -3), (dict(head=4), -3), (dict(stride=-256), -3)]


@pytest.mark.parametrize("kw,code", BAD)
def test_argument_errors(lib, kw, code):
    assert _append(lib, **kw) == code
    assert _attention(lib, **kw) == code
    if not set(kw) & {"stride", "head"}:
        kw = dict(kw)
        ptr = kw.pop("ptr", 256)
        assert lib.moe_kv_read(ptr, ptr, *_structs(**kw), None) == code


def test_attention_argument_errors(lib):
    assert _attention(lib, q_heads=7) == -3          # no multiple of 2 KV heads
    assert _attention(lib, q_heads=0) == -3
    assert _attention(lib, q_heads=2 * 129) == -3    # more than 128 query heads per KV head
    for bad in (0.0, -0.5, float("nan"), float("inf")):
        assert _attention(lib, scale=bad) == -3
    assert _attention(lib, out=None) == -1
    assert _attention(lib, lse=258) == -2


def test_no_structs_is_null(lib):
    c, b = _structs()
    assert lib.moe_kv_append(256, 256, 128, 256, 256, 128, None, b, None) == -1
    assert lib.moe_kv_read(256, 256, c, None, None) == -1


def test_no_tokens_launches_nothing(lib):
    n = lib.moe_launch_count()
    assert _append(lib, T=0, ptr=None) == 0
    assert lib.moe_kv_read(None, None, *_structs(T=0), None) == 0
    assert _attention(lib, T=0, ptr=None, out=None) == 0
    assert lib.moe_launch_count() == n


def test_oracle_e4m3_is_torchs():
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(kv_ref.TABLE))
    assert np.array_equal(t[~np.isnan(t)], kv_ref.TABLE[~np.isnan(t)])
    r = np.random.default_rng(0)
    x = np.concatenate([r.uniform(-448, 448, 20000), r.uniform(-0.05, 0.05, 20000), kv_ref.TABLE[:127],
                        (kv_ref.TABLE[:126] + kv_ref.TABLE[1:127]) / 2])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv_ref.e4m3_codes(x.astype(np.float64)), want)


def test_oracle_scale():
    x = np.array([[448.0, 0], [448.5, 0], [1.75, 0], [1.76, 0], [0, 0], [2.0 ** -140, 0], [-896.0, 1]])
    assert np.array_equal(kv_ref.row_scale(x), [1, 2, 2.0 ** -8, 2.0 ** -7, 1, 2.0 ** -126, 2])


def test_oracle_attention_closed_forms():
    r = np.random.default_rng(1)
    k, v = r.standard_normal((9, 2, 4)), r.standard_normal((9, 2, 4))
    q = r.standard_normal((3, 4, 4))
    # equal scores: the mean of the visible values
    out, lse, _, _ = kv_ref.attention(np.zeros_like(q), k, v, 3, 1.0)
    for i, p in enumerate((6, 7, 8)):
        for h in range(4):
            assert np.allclose(out[i, h], v[:p + 1, h // 2].mean(0)) and np.isclose(lse[i, h], np.log(p + 1))
    # one visible key: its value, whatever the query
    out, lse, _, _ = kv_ref.attention(q, k[:1], v[:1], 1, 0.5)
    assert np.allclose(out[0, 3], v[0, 1]) and np.isclose(lse[0, 3], 0.5 * q[0, 3] @ k[0, 1])
    # no visible key: zero
    out, lse, _, _ = kv_ref.attention(q, k[:1], v[:1], 3, 0.5)
    assert not out[:2].any() and np.isneginf(lse[:2]).all()
