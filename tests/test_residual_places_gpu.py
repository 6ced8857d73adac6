"""Outputs in the place of inputs, one token and two: the same bits as elsewhere; refused over parameters, which stay."""
import pytest

import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.mark.parametrize("H", [1, 64, 384, 2048, 9000, 20000])
@pytest.mark.parametrize("T", [1, 2])
def test_places(T, H):
    import torch

    from bit_mixture_experts_gb300 import MoeError, ResidualNorm
    gen = torch.Generator(device="cuda").manual_seed(H + T)

    def rows(n):
        return torch.randn((n, H), generator=gen, device="cuda").bfloat16()

    x, y, gate = rows(T), rows(T), rows(T)
    w_pre, w_post = rows(1)[0] + 1, rows(1)[0] + 1
    shared = rows(1)[0]
    norm = ResidualNorm(w_pre, w_post, scale=0.9)
    want = [t.clone() for t in norm.add(x, y, gate)]
    for name in ("x", "y", "gate"):
        for place in (0, 1):
            t = dict(x=x.clone(), y=y.clone(), gate=gate.clone())
            if name == "gate" and H == T == 1:
                continue  # (one value, which all tokens may share)
            out = [torch.empty_like(x), torch.empty_like(x)]
            out[place] = t[name]
            got = norm.add(t["x"], t["y"], t["gate"], out=tuple(out))
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (name, place)
    if T > 1:
        return
    kept = [p.clone() for p in (w_pre, w_post, shared)]
    for p in (w_pre, w_post, shared):
        for place in (0, 1):
            out = [torch.empty_like(x), torch.empty_like(x)]
            out[place] = p.view(1, H)
            with pytest.raises(MoeError, match="OVERLAP"):
                norm.add(x, y, shared, out=tuple(out))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((w_pre, w_post, shared), kept))
