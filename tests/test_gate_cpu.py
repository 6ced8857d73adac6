"""The gates' and residual norms' oracle against independent forms, and the argument errors of their entry points (found
on the host before any CUDA call).  No compute runs on a GPU."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import gate_ref, moe_ref


@pytest.fixture(scope="module")
def lib():
    from bit_mixture_experts_gb300 import _lib, build
    build.build()
    return _lib.load()


# --------------------------------------------------------------------------- #
# oracle
# --------------------------------------------------------------------------- #
def test_softmax_gate_without_more_is_the_plain_router():
    l = np.random.default_rng(0).standard_normal((40, 24)).astype(np.float32)
    ids, w = gate_ref.choose(l, 5)
    ref_ids, ref_w = moe_ref.topk_route(l, 5)
    np.testing.assert_array_equal(ids, ref_ids)
    np.testing.assert_allclose(w, ref_w, rtol=1e-6)


def test_choice_by_hand():
    # scores 1/2, 3/4, 1/4, 1/2: logits 0, ln 3, -ln 3, 0
    l = np.log(np.array([1.0, 3.0, 1 / 3, 1.0]))
    ids, w = gate_ref.choose_token(l, 2, "sigmoid", renorm=False)
    assert ids.tolist() == [1, 0] and np.allclose(w, [0.75, 0.5])
    b = [0.0, -0.5, 0.3, 0.0]  # values 0.5, 0.25, 0.55, 0.5: the bias chooses, the score weighs
    ids, w = gate_ref.choose_token(l, 3, "sigmoid", b, scale=2.0)
    assert ids.tolist() == [2, 0, 3] and np.allclose(w, 2 * np.array([0.25, 0.5, 0.5]) / 1.25)
    # groups {0, 1} and {2, 3}: by their largest the second one, by the sum of two the second too, without bias the first
    assert gate_ref.choose_token(l, 1, "sigmoid", b, 2, 1, "max")[0].tolist() == [2]
    assert gate_ref.choose_token(l, 2, "sigmoid", b, 2, 1, "top2")[0].tolist() == [2, 3]
    assert gate_ref.choose_token(l, 2, "sigmoid", None, 2, 1, "top2")[0].tolist() == [1, 0]
    # largest and sum disagree: 0.9 + 0.1 and 0.6 + 0.6
    l = np.log(np.array([9.0, 1 / 9, 1.5, 1.5]))
    assert gate_ref.choose_token(l, 1, "sigmoid", None, 2, 1, "max")[0].tolist() == [0]
    assert gate_ref.choose_token(l, 1, "sigmoid", None, 2, 1, "top2")[0].tolist() == [2]
    # softmax scores over all experts, not over the chosen
    ids, w = gate_ref.choose_token(np.log([1.0, 2.0, 5.0]), 2, "softmax", renorm=False)
    assert ids.tolist() == [2, 1] and np.allclose(w, [5 / 8, 2 / 8])


def test_experts_that_are_not_available_by_hand():
    n = -np.inf
    ids, w = gate_ref.choose_token([n, 0.0, np.nan, n], 3, "sigmoid")
    assert ids.tolist() == [1, 0, 2] and w.tolist() == [1.0, 0.0, 0.0]
    ids, w = gate_ref.choose_token([n] * 4, 2, "softmax", [1.0, 2.0, 3.0, 4.0])
    assert ids.tolist() == [0, 1] and w.tolist() == [0.0, 0.0]
    # a group with one is scored by it; one without any is behind a group of negative values
    ids, _ = gate_ref.choose_token([n, 2.0, 0.0, 0.0, n, n], 2, "sigmoid", [0.0] + [-9.0] * 5, 3, 2, "top2")
    assert ids.tolist() == [1, 2]


def test_many_tokens_at_a_time_are_the_same():
    r = np.random.default_rng(2)
    l, b = r.standard_normal((30, 48)), r.standard_normal(48) * 0.05
    l[:10] = np.round(l[:10] * 2) / 2
    for score in ("softmax", "sigmoid"):
        for bias in (None, b):
            for groups, top, how in ((1, None, "max"), (6, 2, "max"), (6, 2, "top2"), (6, 6, "top2")):
                kw = dict(score=score, bias=bias, groups=groups, top_groups=top, group_score=how, scale=1.5)
                one, many = gate_ref.choose(l, 7, **kw), gate_ref.choose_many(l, 7, **kw)
                np.testing.assert_array_equal(one[0], many[0])
                np.testing.assert_allclose(one[1], many[1], rtol=1e-14)


def _residual_fractions(x, y, w_pre, w_post, gate, scale, eps, offset):
    """The definition with exact sums of squares."""
    def rms(v):
        return math.sqrt(float(sum(Fraction(float(a)) ** 2 for a in v) / len(v)) + eps)
    z = [a / rms(y) * (w + offset) for a, w in zip(y, w_post)]
    r = [scale * a + g * b for a, g, b in zip(x, gate, z)]
    return r, [a / rms(r) * (w + offset) for a, w in zip(r, w_pre)]


def test_residual_oracle_against_exact_sums():
    rng = np.random.default_rng(4)
    x, y, a, b, g = rng.standard_normal((5, 33))
    r, n = _residual_fractions(x, y, a, b, g, 0.75, 1e-3, 1.0)
    got = gate_ref.residual(x[None], y[None], a, b, g, 0.75, 1e-3, 1.0)
    np.testing.assert_allclose(got[0][0], r, rtol=1e-13)
    np.testing.assert_allclose(got[1][0], n, rtol=1e-13)


def test_residual_bounds_hold_for_float32_and_no_more():
    """A float32 emulation stays within the bounds; one that rounds the normed y to bf16 on the way does not."""
    rng = np.random.default_rng(7)
    x, y = (rng.standard_normal((20, 512)).astype(np.float32) for _ in range(2))
    w = rng.standard_normal(512).astype(np.float32)
    f = np.float32

    def run(rounded):
        z = y / np.sqrt((y * y).mean(1, dtype=f, keepdims=True) + f(1e-6)) * w
        if rounded:
            z = moe_ref.round_bf16(z).astype(f)
        r = x + z
        return r, r / np.sqrt((r * r).mean(1, dtype=f, keepdims=True) + f(1e-6)) * w

    want = gate_ref.residual(x, y, w, w)
    for rounded in (False, True):
        r, n = run(rounded)
        inside = (np.abs(r - want[0]) <= want[2]).all() and (np.abs(n - want[1]) <= want[3]).all()
        assert inside == (not rounded)


# --------------------------------------------------------------------------- #
# argument errors: -1 NULL, -2 ALIGN, -3 SHAPE, -4 WORKSPACE, -7 MODE, -8 OVERLAP
# --------------------------------------------------------------------------- #
def _gate(lib, T=8, E=16, k=2, ptr=16, ws=None, no_gate=False, **kw):
    from bit_mixture_experts_gb300 import _lib
    f = dict(bias=None, score=1, groups=1, top_groups=1, group_score=1, renorm=1, scale=1.0)
    f.update(kw)
    g = None if no_gate else _lib.Gate(*f.values())
    if ws is None:
        return lib.moe_gate(ptr, T, E, k, g, ptr, ptr, None)
    return lib.moe_route_gated(ptr, T, E, k, g, 64, *([ptr or 16] * 8), ptr, ws, None)


@pytest.mark.parametrize("route", [False, True])
def test_gate_argument_errors(lib, route):
    def call(**kw):
        return _gate(lib, ws=1 << 20 if route else None, **kw)
    assert call(no_gate=True) == -1
    assert call(score=2) == -7 and call(score=-1) == -7 and call(group_score=2) == -7
    assert call(groups=0) == -3 and call(groups=33, E=33) == -3 and call(groups=3, top_groups=1) == -3
    assert call(groups=4, top_groups=0) == -3 and call(groups=4, top_groups=5) == -3
    assert call(groups=8, top_groups=1, k=3) == -3  # two experts stay
    assert call(scale=float("inf")) == -3 and call(scale=float("nan")) == -3
    assert call(bias=18) == -2
    assert call(T=-1) == -3 and call(T=(1 << 20) + 1) == -3 and call(E=1025) == -3 and call(k=33, E=64) == -3
    assert call(k=17) == -3 and call(k=0) == -3
    assert call(ptr=8) == -2
    if route:
        assert call(T=0) == -3
        assert _gate(lib, T=4096, ws=0) == -4
    else:
        assert call(ptr=None) == -1
        assert call(T=0, ptr=None) == 0  # does nothing


@pytest.mark.parametrize("route", [False, True])
def test_a_gates_outputs_lie_apart(lib, route):
    """T 8, E 16, k 2: logits 512 bytes, ids and weights 64, bias 64."""
    from bit_mixture_experts_gb300 import _lib

    def call(logits=BASE, ids=2 * BASE, w=3 * BASE, bias=4 * BASE, **kw):
        g = _lib.Gate(bias, 1, 1, 1, 1, 1, 1.0)
        if not route:
            return lib.moe_gate(logits, 8, 16, 2, g, ids, w, None)
        return lib.moe_route_gated(logits, 8, 16, 2, g, 64, ids, w, *([9 * BASE] * 6), 9 * BASE, 1 << 20, None)
    assert call(ids=BASE) == -8 and call(w=BASE + 512 - 16) == -8 and call(ids=BASE - 48) == -8
    assert call(ids=3 * BASE) == -8 and call(w=2 * BASE + 48) == -8
    assert call(w=4 * BASE) == -8 and call(ids=4 * BASE + 48) == -8 and call(bias=3 * BASE - 60) == -8


BASE = 1 << 20  # addresses that no call gets to follow


def _residual(lib, T=4, H=64, y=BASE, y_stride=None, k=0, none=False, **kw):
    from bit_mixture_experts_gb300 import _lib
    f = dict(x=2 * BASE, x_stride=H, r=3 * BASE, r_stride=H, n=4 * BASE, n_stride=H, w_pre=5 * BASE, w_post=6 * BASE,
             gate=None, gate_token_stride=0, gate_per_channel=0, post=1, stream_f32=0, param_f32=0, gate_f32=0,
             offset=0.0, scale=1.0, eps=1e-6)
    f.update(kw)
    p = None if none else _lib.Residual(*f.values())
    if k:
        return lib.moe_combine_residual_norm(y, 7 * BASE, 8 * BASE, T, H, k, p, None)
    return lib.moe_residual_norm(y, H if y_stride is None else y_stride, T, H, p, None)


@pytest.mark.parametrize("k", [0, 2])
def test_residual_argument_errors(lib, k):
    def call(**kw):
        return _residual(lib, k=k, **kw)
    assert call(none=True) == -1
    assert call(T=-1) == -3 and call(T=(1 << 20) + 1) == -3 and call(H=0) == -3 and call(H=32769) == -3
    assert call(T=0) == 0
    assert call(x_stride=-1) == -3 and call(gate_token_stride=-64) == -3 and call(x_stride=1 << 40) == -3
    assert call(r_stride=63) == -3 and call(n_stride=0) == -3
    for name in ("eps", "scale", "offset"):
        assert call(**{name: float("nan")}) == -3 and call(**{name: float("inf")}) == -3
    assert call(eps=-1e-6) == -3
    assert call(x=None) == -1 and call(r=None, n=None) == -1
    assert call(x=2 * BASE + 1) == -2 and call(x=2 * BASE + 2, stream_f32=1) == -2
    assert call(r=3 * BASE + 2, stream_f32=1) == -2 and call(n=4 * BASE + 1) == -2
    assert call(w_pre=5 * BASE + 2, param_f32=1) == -2 and call(w_post=6 * BASE + 1) == -2
    assert call(gate=7 * BASE + 2, gate_f32=1) == -2
    # outputs over one another, over inputs that other rows read, or not quite in an input's place
    row = 2 * 64
    assert call(n=3 * BASE) == -8 and call(n=3 * BASE + 3 * row) == -8
    assert call(r=2 * BASE + row) == -8 and call(r=2 * BASE, r_stride=72) == -8
    assert call(r=2 * BASE, stream_f32=1, r_stride=64, n=2 * BASE) == -8
    assert call(n=2 * BASE, stream_f32=1) == -8  # bf16 over a float32 stream
    assert call(r=5 * BASE) == -8 and call(n=6 * BASE + row - 2) == -8
    assert call(n=BASE - row) == -8
    assert call(gate=7 * BASE, r=7 * BASE) == -8  # a gate for all tokens
    if k:
        assert call(r=BASE) == -8 and call(n=BASE + 11 * row) == -8  # rows that other tokens read
        assert call(y=None) == -1 and call(y=BASE + 2) == -2
        assert call(r=7 * BASE - 2 * row) == -8 and call(n=8 * BASE) == -8  # over the rows' places and weights
        assert lib.moe_combine_residual_norm(BASE, BASE, BASE, 4, 64, 33, None, None) == -3
    else:
        assert call(y_stride=-1) == -3
        assert call(x_stride=0, r=2 * BASE) == -8  # one row of x for all tokens


def test_overlap_of_columns(lib):
    """Columns of one wider tensor: interleaved rows that share no byte pass the check (the call then ends where it looks
    for a device: there is none here), shifted ones that do are refused."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    wide = dict(x_stride=192, r_stride=192, n_stride=192, x=2 * BASE)
    assert _residual(lib, r=2 * BASE + 128, n=2 * BASE + 256, **wide) == -5
    assert _residual(lib, r=2 * BASE, n=2 * BASE + 256, **wide) == -5
    assert _residual(lib, r=2 * BASE - 128, n=2 * BASE + 128, **wide) == -5
    assert _residual(lib, r=2 * BASE + 126, n=2 * BASE + 256, **wide) == -8
    assert _residual(lib, r=2 * BASE + 258, n=8 * BASE, **wide) == -8  # reaches into x's next row
    assert _residual(lib, r=2 * BASE - 126, n=8 * BASE, **wide) == -8


def test_layer_gated_argument_errors(lib):
    from bit_mixture_experts_gb300 import _lib
    P = 16
    gate = _lib.Gate(None, 1, 1, 1, 1, 1, 1.0)

    def call(T=4, H=128, E=16, k=2, block_n=8, logits=P, gate=gate, out=P, residual=None, weights=True, **buf):
        f = {n: P for n, _ in _lib.Buffers._fields_}
        f.update(workspace_bytes=1 << 20, decode_ws_bytes=1 << 20, combine_ws_bytes=1 << 20, **buf)
        return lib.moe_layer_forward_gated(P, logits, gate, out, residual, T, H, 128, E, k, block_n, 0,
                                           _lib.Weights(P, P) if weights else None, _lib.Buffers(**f), None)
    assert call(weights=False) == -1
    assert call(gate=None) == -1
    assert call(gate=_lib.Gate(None, 5, 1, 1, 1, 1, 1.0)) == -7
    assert call(logits=8) == -2
    assert call(out=None) == -1
    assert call(H=100) == -3
    bad = _lib.Residual(x=P, r=P, x_stride=128, r_stride=128, eps=-1.0)
    assert call(residual=bad) == -3
    over = _lib.Residual(x=2 * BASE, r=16 + 256 * 5, x_stride=128, r_stride=128)  # a row of y
    assert call(residual=over) == -8
    assert call(residual=_lib.Residual(x=P, x_stride=128)) == -1


def test_python_checks():
    import torch

    from bit_mixture_experts_gb300 import ExpertGate, ResidualNorm
    with pytest.raises(ValueError, match="score"):
        ExpertGate(2, "tanh")
    with pytest.raises(ValueError, match="group_score"):
        ExpertGate(2, group_score="mean")
    for b in (torch.zeros(8), torch.zeros(8, dtype=torch.float64), torch.zeros((2, 4))):
        with pytest.raises(ValueError, match="bias"):
            ExpertGate(2, bias=b)
    for l in (torch.zeros((2, 8)), torch.zeros(8)):
        with pytest.raises(ValueError, match="logits"):
            ExpertGate(2).choose(l)
    for w in (torch.ones(8), torch.ones((2, 4)), torch.ones(8, dtype=torch.float16)):
        with pytest.raises(ValueError, match="w_pre"):
            ResidualNorm(w)
    with pytest.raises(ValueError, match="x must be"):
        ResidualNorm().norm(torch.zeros((2, 8)))
    with pytest.raises(ValueError, match="x must be"):
        ResidualNorm().add(torch.zeros(8), torch.zeros(8))


def test_what_the_library_was_told_is_fixed():
    """A tensor put in a gain's or a bias's place would not be read: the calls would go on with the old one's memory."""
    import torch

    from bit_mixture_experts_gb300 import ExpertGate, ResidualNorm
    gate, norm = ExpertGate(2), ResidualNorm(scale=0.5)
    for obj, name in [(gate, n) for n in ("bias", "k", "scale", "renorm", "score", "groups", "top_groups", "group_score")] + [
            (norm, n) for n in ("w_pre", "w_post", "scale", "eps", "offset")]:
        with pytest.raises(AttributeError, match="fixed"):
            setattr(obj, name, torch.zeros(8))
    assert gate.bias is None and norm.scale == 0.5
