"""What the decoder block and its serving loop refuse before they do anything, without a GPU."""
import types

import pytest

torch = pytest.importorskip("torch")

H = 8


def _serve(lens, chunk, steps):
    from bit_mixture_experts_gb300 import block
    cache = types.SimpleNamespace(page_size=16, num_pages=64, batch=lambda *a: None)
    stub = types.SimpleNamespace(cache=cache, forward=lambda x, batch: x)
    return block.serve(stub, [torch.zeros((n, H)) for n in lens], chunk, steps)


def test_serve_counts():
    sizes = [new for _, new, _, _, _ in _serve((5, 2), 3, 2)]
    assert sizes == [[3, 2], [2, 0], [1, 1], [1, 1]]
    assert list(_serve((1,), 3, 0))[0][1] == [1]


@pytest.mark.parametrize("lens,chunk,steps", [((3, 0), 2, 1), ((0,), 2, 0), ((3,), 0, 1), ((3,), -1, 1), ((3,), 2, -1),
                                              ((), 2, 1)])
def test_serve_refuses_what_it_cannot_serve(lens, chunk, steps):
    with pytest.raises(ValueError):
        next(_serve(lens, chunk, steps))


@pytest.mark.parametrize("q_heads,kv_heads,extra", [(4, 2, 1), (3, 2, 0)])
def test_block_refuses_projections_that_are_no_heads(q_heads, kv_heads, extra):
    """w_o of no whole number of heads, and query heads that the KV heads cannot be shared out to."""
    from bit_mixture_experts_gb300 import block
    d, E = 64, 4
    moe, cache = types.SimpleNamespace(H=H, E=E), types.SimpleNamespace(d=d, heads=kv_heads)
    w = [torch.zeros(s) for s in (((q_heads + 2 * kv_heads) * d, H), (H, q_heads * d + extra), (E, H))]
    with pytest.raises(ValueError, match="q_heads"):
        block.DecoderBlockW4(*w, moe, cache)
    ok = [torch.zeros(s) for s in ((8 * d, H), (H, 4 * d), (E, H))]
    assert block.DecoderBlockW4(*ok, moe, types.SimpleNamespace(d=d, heads=2)).q_heads == 4


def test_block_takes_three_norms():
    from bit_mixture_experts_gb300 import block
    d, E = 64, 4
    moe, cache = types.SimpleNamespace(H=H, E=E), types.SimpleNamespace(d=d, heads=2)
    w = [torch.zeros(s) for s in ((8 * d, H), (H, 4 * d), (E, H))]
    with pytest.raises(ValueError, match="three norms"):
        block.DecoderBlockW4(*w, moe, cache, norms=(None, None))
