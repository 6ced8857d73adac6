"""What the decoder block's serving loop refuses before it does anything, without a GPU."""
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

