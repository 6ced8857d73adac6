"""Whose place a residual norm's outputs may take, with one token as with many: its own rows', never those of parameters.
The addresses are made up; a call that passes ends where it looks for a device (-5), one that is refused before (-8)."""
import pytest

torch = pytest.importorskip("torch")

from test_gate_cpu import BASE, _residual, lib  # noqa: F401  (a fixture)

GATE = 9 * BASE


@pytest.mark.parametrize("H", [1, 64, 384, 9000])
@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("k", [0, 2])
def test_places(lib, T, H, k):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")

    def call(**kw):
        f = dict(gate=GATE, gate_token_stride=0, gate_per_channel=1)
        f.update(kw)
        return _residual(lib, T=T, H=H, k=k, **f)

    assert call() == -5
    for out in ("r", "n"):
        assert call(**{out: 5 * BASE}) == -8 and call(**{out: 6 * BASE}) == -8  # gains
        assert call(**{out: GATE}) == -8                                        # a gate of all tokens
        assert call(**{out: GATE}, gate_per_channel=0) == -8                    # one value of all tokens
        assert call(**{out: GATE}, gate_token_stride=H) == -5                   # a gate per token and channel
        assert call(**{out: GATE + 2}, gate_token_stride=H) == (-8 if H > 1 or T > 1 else -5)
        if H > 1:
            assert call(**{out: GATE}, gate_token_stride=H, gate_per_channel=0) == -8  # a value per token
        assert call(**{out: 2 * BASE}) == -5                                    # x
        assert call(**{out: BASE}) == (-8 if k else -5)                         # y; the rows that a combine gathers


def test_a_token_s_own_gate_is_told_apart():
    """What the library is told of [H], [1, H], [1, 1] and [T, H] gates."""
    from bit_mixture_experts_gb300 import residual

    class Cuda(torch.Tensor):  # a tensor that says it is on the device
        is_cuda = True

    def described(T, gate, H=64):
        norm = residual.ResidualNorm.__new__(residual.ResidualNorm)
        object.__setattr__(norm, "H", None)
        object.__setattr__(norm, "_constants", residual._lib.Residual())
        x = torch.zeros((T, H)).as_subclass(Cuda)
        s, _ = norm.describe(x, gate, (x, None))
        return s.gate_token_stride, s.gate_per_channel

    before = residual._current_device
    residual._current_device = lambda: None
    try:
        z = torch.zeros
        assert described(1, z(64)) == (0, 1) and described(5, z(64)) == (0, 1)
        assert described(1, z((1, 64))) == (64, 1) and described(5, z((1, 64))) == (0, 1)
        assert described(1, z((1, 1))) == (0, 0) and described(5, z((5, 1))) == (1, 0) and described(5, z((1, 1))) == (0, 0)
        assert described(5, z((5, 64))) == (64, 1) and described(1, z((1, 128))[:, :64]) == (128, 1)
        assert described(1, z(64).expand(1, 64))[1] == 1 and described(5, z(64).expand(5, 64)) == (0, 1)
    finally:
        residual._current_device = before
