"""moe_gate and moe_route_gated on the GPU against the float64 oracle: the same experts in the same order, always;
weights within the error of their FP32 arithmetic."""
import numpy as np
import pytest

from oracle import gate_ref, moe_ref

pytestmark = pytest.mark.gpu


def setup_module():
    import gpu_util
    gpu_util.ensure_built()


def make(k, bias=None, **kw):
    import torch

    from bit_mixture_experts_gb300 import ExpertGate
    return ExpertGate(k, bias=None if bias is None else torch.tensor(bias, dtype=torch.float32, device="cuda"), **kw)


def weight_bound(ref, logits, ids, kw):
    """u = 2^-24.  A score: exp 4 u, its argument's rounding u (top - l), sum and division 3 u.  The sum over the experts
    (at most 64 per lane, then 5 steps): 69 u, its terms 4 u and as much as ln E u for their arguments; the sum over the
    chosen 5 u and its terms' error; division and scale 2 u.  Below 2^-126 scores are flushed."""
    l = np.take_along_axis(np.minimum(np.nan_to_num(logits, nan=-np.inf, posinf=3.4e38), 3.4e38), ids, 1)
    top = np.nanmax(np.where(np.isfinite(logits), logits, np.nan), axis=1, initial=0, keepdims=True)
    rel = 2 * 7 + 7.0
    if kw.get("score", "softmax") == "softmax":
        with np.errstate(invalid="ignore"):
            rel = rel + np.where(np.isfinite(l), np.abs(top - l), 0) + 80
    return np.abs(ref) * rel * 2.0 ** -24 + abs(kw.get("scale", 1.0)) * 2.0 ** -120


def check(logits, k, bias=None, **kw):
    import torch

    from bit_mixture_experts_gb300 import _lib
    gate = make(k, bias, **kw)
    T, E = logits.shape
    # guard rows behind the last token stay as they are
    ids = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    gate.choose(torch.tensor(logits, dtype=torch.float32, device="cuda"), out=(ids[:T], w[:T]))
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 0
    assert (ids[T] == -7).all() and (w[T] == -7).all()
    want_ids, want_w = gate_ref.choose(logits.astype(np.float32), k, bias=None if bias is None else np.float32(bias), **kw)
    np.testing.assert_array_equal(ids[:T].cpu().numpy(), want_ids)
    got = w[:T].double().cpu().numpy()
    off = np.abs(got - want_w) - weight_bound(want_w, logits.astype(np.float64), want_ids, kw)
    assert (off <= 0).all(), (off.max(), np.abs(got - want_w).max())


def draw(T, E, seed, coarse=False):
    r = np.random.default_rng(seed)
    l = (r.standard_normal((T, E)) * np.exp(0.3 * r.standard_normal((T, 1))) + 0.7 * r.standard_normal(E)).astype(np.float32)
    if coarse:
        l = np.round(l * 4) / 4
    return l, (np.round(r.standard_normal(E) * 40) * 0.001).astype(np.float32)


CASES = [  # T, E, k, groups, top_groups
    (1, 1, 1, 1, 1), (3, 2, 2, 1, 1), (5, 7, 3, 1, 1), (33, 32, 32, 1, 1), (9, 37, 5, 1, 1), (17, 74, 8, 2, 1),
    (64, 160, 6, 8, 3), (333, 256, 8, 8, 4), (100, 256, 8, 1, 1), (7, 96, 32, 3, 2), (8, 1020, 16, 17, 5),
    (5, 1000, 4, 5, 2), (4, 1024, 32, 32, 9), (3, 1024, 32, 1, 1), (2, 64, 4, 32, 2), (6, 1023, 31, 31, 3),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,groups,top", CASES)
def test_choice_and_weights(T, E, k, groups, top, with_bias, score):
    seed = T * 1000 + E + 7 * k + 13 * groups
    for i, (group_score, renorm, coarse) in enumerate([("top2", True, False), ("max", False, True)]):
        l, b = draw(T, E, seed + i, coarse)
        check(l, k, b if with_bias else None, score=score, groups=groups, top_groups=top, group_score=group_score,
              renorm=renorm, scale=2.5 if renorm else 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_scores_go_to_the_lower_index(score):
    E = 256
    flat = np.zeros((4, E), np.float32)
    check(flat, 8, score=score)
    check(flat, 8, np.zeros(E), score=score, groups=8, top_groups=4)
    b = np.zeros(E)
    b[[3, 77, 78, 200, 255]] = 0.001
    check(flat, 8, b, score=score, groups=8, top_groups=4)
    check(np.where(np.arange(E) % 2, 0.0, -0.0)[None].astype(np.float32), 9, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(1, 1), (8, 3)])
def test_scores_that_differ_by_less_than_32_bits_hold(score, groups, top):
    # biases that bring every expert's value to the same number, as far as 32 bits go: the order is that of what is left
    E, r = 256, np.random.default_rng(5)
    l = r.standard_normal((1, E)).astype(np.float32)
    s, _ = gate_ref.scores(l[0], score)
    b = (0.9 - s).astype(np.float32)
    check(np.repeat(l, 3, 0), 8, b, score=score, groups=groups, top_groups=top)
    check(np.repeat(l, 3, 0), 32, b, score=score, groups=groups, top_groups=max(top, 4) if groups > 1 else 1,
          group_score="max")
    # only the border of the choice is near: expert k is next to expert k + 1
    l = np.linspace(3, -3, E).astype(np.float32)[None]
    s, _ = gate_ref.scores(l[0], score)
    b = np.zeros(E, np.float32)
    b[200] = np.float32(s[7] - s[200])
    check(l, 8, b, score=score)
    check(l, 9, b, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_experts_that_are_not_available(score, with_bias, group_score):
    l, b = draw(12, 64, 3)
    b = b if with_bias else None
    l[0] = -np.inf
    l[1, :] = np.nan
    l[2, 10:] = -np.inf
    l[3, ::2] = np.nan
    l[4, 8:16] = -np.inf   # a group without any
    l[5, np.arange(64) % 8 != 3] = -np.inf  # one in each group
    l[6, 5] = np.inf
    l[7, [5, 9]] = np.inf
    l[8, :60] = -np.inf
    l[9] = -200.0  # scores that 32 bits do not hold (sigmoid)
    for groups, top in ((1, 1), (8, 2)):
        check(l, 8, b, score=score, groups=groups, top_groups=top, group_score=group_score)


def test_large_logits():
    r = np.random.default_rng(1)
    l = (r.standard_normal((16, 128)) * 60).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        check(l, 4, None, score=score)
        check(l, 4, np.zeros(128), score=score, groups=4, top_groups=2) if score == "softmax" else None


def test_no_tokens():
    import torch
    ids, w = make(2).choose(torch.empty((0, 16), device="cuda"))
    assert ids.shape == (0, 2) and w.shape == (0, 2)


def test_softmax_gate_is_moe_route():
    import torch

    from bit_mixture_experts_gb300 import _lib
    for T, E, k in ((5, 16, 2), (300, 256, 8)):
        l = torch.tensor(draw(T, E, T)[0], device="cuda")
        got = make(k).route(l, 32)
        ref = [torch.empty_like(t) for t in got]
        ws = torch.zeros(max(16, _lib.moe_route_workspace_size(T, E, k, 32)), dtype=torch.uint8, device="cuda")
        _lib.moe_route(l, k, 32, *ref, ws)
        n = int(ref[7])
        for name, a, b in zip(got._fields, got, ref):
            a, b = (a[:n], b[:n]) if name == "block_map" else (a, b)
            assert torch.equal(a, b), name


@pytest.mark.parametrize("T,E,k,block_n,how", [
    (33, 40, 32, 8, "any"), (1023, 256, 8, 64, "any"), (1024, 256, 8, 64, "one"), (2047, 7, 4, 16, "twice"),
    (4096, 600, 2, 32, "any"), (9000, 1024, 1, 128, "any"), (16383, 256, 8, 64, "few"), (16384, 256, 8, 64, "any"),
    (70001, 33, 5, 8, "few"), (140000, 64, 1, 64, "one")])
def test_route_of_experts_chosen_already(T, E, k, block_n, how):
    """Around the sizes where the rounds of a chunk begin and its CTAs change; experts without any and with all tokens."""
    import torch

    from bit_mixture_experts_gb300 import _lib
    rng = np.random.default_rng(T)
    ids = rng.integers(0, E, (T, k))
    if how == "one":
        ids[:] = E - 1
    if how == "twice":
        ids[:, 1:] = ids[:, :1]
    if how == "few":
        ids = np.where(rng.random((T, k)) < 0.9, E // 2, ids)
    dev = "cuda"
    want = gate_ref.sort_assignments(ids, E)
    tiles = moe_ref.block_map(want[0], want[1], T, block_n)
    given = torch.from_numpy(ids.astype(np.int32)).to(dev)
    w = torch.full((T, k), 7.0, device=dev)
    out = [torch.full(n, -9, dtype=torch.int32, device=dev) for n in
           ((E,), (E + 1,), (T * k,), (T * k,), (_lib.moe_block_map_capacity(T, E, k, block_n), 3), (1,))]
    ws = torch.zeros(_lib.moe_route_workspace_size(T, E, k, block_n), dtype=torch.uint8, device=dev)
    for _ in range(2):  # the second call finds the scratch as the first left it
        _lib.moe_route_gated(None, T, E, k, None, block_n, given, w, *out, ws)
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 0
    for name, got, ref in zip(("counts", "offsets", "perm", "inv_perm"), out, want):
        np.testing.assert_array_equal(got.cpu().numpy(), ref, err_msg=name)
    assert int(out[5]) == len(tiles)
    got = out[4].cpu().numpy()
    np.testing.assert_array_equal(got[:len(tiles)], tiles)
    assert (got[len(tiles):] == -9).all()
    assert (given.cpu().numpy() == ids).all() and (w == 7).all()


@pytest.mark.parametrize("T,E,k,block_n", [(1, 256, 8, 8), (100, 64, 4, 16), (129, 64, 8, 64), (3000, 256, 8, 64)])
def test_route(T, E, k, block_n):
    import torch

    from bit_mixture_experts_gb300 import _lib
    l, b = draw(T, E, T + E)
    kw = dict(score="sigmoid", groups=8, top_groups=4, scale=2.5)
    gate = make(k, b, **kw)
    lt = torch.tensor(l, device="cuda")
    got = [gate.route(lt, block_n) for _ in range(2)][1]  # the second call finds the scratch as the first left it
    ids, w = gate.choose(lt)
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 0
    assert torch.equal(got.topk_ids, ids) and torch.equal(got.topk_w, w)
    want = gate_ref.sort_assignments(ids.cpu().numpy(), E)
    for name, ref in zip(("counts", "offsets", "perm", "inv_perm"), want):
        np.testing.assert_array_equal(getattr(got, name).cpu().numpy(), ref, err_msg=name)


def test_streams_and_graphs():
    import torch
    gate = make(8, draw(1, 256, 9)[1], score="sigmoid", groups=8, top_groups=4)
    a, b = (torch.tensor(draw(700, 256, s)[0], device="cuda") for s in (1, 2))
    want = [gate.route(x, 64) for x in (a, b)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        got = gate.route(b, 64, stream=s)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got[:6], want[1][:6]))
    # two graphs captured on one stream, replayed together with other calls in between
    x = a.clone()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(gate.route(x, 64))
        graphs.append(g)
    x.copy_(b)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs[0].replay()
    with torch.cuda.stream(other):
        graphs[1].replay()
    gate.route(a, 64)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(o[:6], want[1][:6]))
    # the bias is read by every call
    gate.bias.zero_()
    ids, _ = gate.choose(b)
    np.testing.assert_array_equal(
        ids.cpu().numpy(), gate_ref.choose(b.cpu().numpy(), 8, score="sigmoid", bias=np.zeros(256), groups=8, top_groups=4)[0])


MANY = [  # T, E, k, groups, top_groups: tokens enough that a warp takes two or four together, in every width of a lane
    (4001, 256, 8, 8, 4), (9001, 256, 8, 8, 4), (9002, 256, 8, 1, 1), (8003, 160, 6, 8, 3), (8001, 64, 8, 4, 2),
    (7500, 256, 16, 8, 4), (7501, 256, 20, 8, 4), (9003, 128, 4, 16, 5), (8002, 252, 8, 9, 4), (8000, 255, 6, 17, 5),
    (7777, 96, 8, 32, 7), (4100, 512, 16, 16, 4), (8004, 512, 8, 1, 1), (4000, 1000, 8, 5, 2), (20000, 37, 2, 1, 1),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top", MANY)
def test_many_tokens(T, E, k, groups, top, score):
    import torch

    from bit_mixture_experts_gb300 import _lib
    for i, (with_bias, how, coarse) in enumerate(((True, "top2", False), (False, "top2", True), (True, "max", True),
                                                  (False, "max", False))):
        l, b = draw(T, E, T + 10 * i, coarse)
        if i == 2:  # many values that 32 bits do not tell apart
            s, _ = gate_ref.scores(l[0], score)
            b = (0.5 - s).astype(np.float32)
            l[::7] = l[0]
        b = b if with_bias else None
        kw = dict(score=score, groups=groups, top_groups=top, group_score=how, renorm=i % 2 == 0, scale=2.0)
        gate = make(k, b, **kw)
        ids, w = gate.choose(torch.tensor(l, device="cuda"))
        torch.cuda.synchronize()
        assert _lib.moe_get_device_error() == 0
        want_ids, want_w = gate_ref.choose_many(l, k, bias=b, **kw)
        np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
        off = np.abs(w.double().cpu().numpy() - want_w) - weight_bound(want_w, l.astype(np.float64), want_ids, kw)
        assert (off <= 0).all(), off.max()


def test_unavailable_experts_among_many_tokens():
    """Tokens of one warp with and without experts that are not available."""
    import torch
    l, b = draw(8100, 256, 1)
    r = np.random.default_rng(0)
    l[::3, r.permutation(256)[:40]] = -np.inf
    l[5::97] = np.nan
    l[8::101, :250] = -np.inf
    kw = dict(score="sigmoid", groups=8, top_groups=4, scale=2.5)
    ids, w = make(8, b, **kw).choose(torch.tensor(l, device="cuda"))
    few, few_w = make(8, b, **kw).choose(torch.tensor(l[:700], device="cuda"))  # a token a warp
    assert torch.equal(ids[:700], few) and torch.equal(w[:700], few_w)
    at = np.r_[0:60, 8000:8100, 5:8100:97][:200]
    want_ids, want_w = gate_ref.choose(l[at], 8, bias=b, **kw)
    np.testing.assert_array_equal(ids.cpu().numpy()[at], want_ids)
    np.testing.assert_allclose(w.double().cpu().numpy()[at], want_w, rtol=2e-6)


def test_a_bias_out_of_proportion():
    """Biases that switch experts on and off: the range of values is no longer that of the scores."""
    l, b = draw(60, 256, 4)
    b[[3, 50, 51, 200]] = [1000.0, -1000.0, 1e6, -1e6]
    for kw in (dict(), dict(groups=8, top_groups=4), dict(groups=8, top_groups=3, group_score="max")):
        for score in ("sigmoid", "softmax"):
            check(l, 8, b, score=score, **kw)
