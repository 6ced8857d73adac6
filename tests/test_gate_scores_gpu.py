"""Gates where scores are next to 0 or to 1: renormalised weights are the ratios of the scores however small those are,
and the choice holds to 2^-40 where the scores are closer than that."""
import numpy as np
import pytest

from oracle import gate_ref
from test_gate_gpu import make

pytestmark = pytest.mark.gpu

# u = 2^-24.  A score over the largest one: exp and the rest of its argument's difference 6 u, 1 + exp 3 u (its exp is at
# most the half), division 1 u; the sum over the chosen the same and 5 u; division and scale 2 u.
REL = 27 * 2.0 ** -24
TOL = 2.0 ** -40  # of the values that are compared


def setup_module():
    import gpu_util
    gpu_util.ensure_built()


def tokens(E, seed=0):
    """Logits, a row each."""
    r = np.random.default_rng(seed)
    flat = [np.full(E, x) for x in (-87.5, -88.0, -88.5, -100.0, -200.0, -3e38)]
    rows = flat + [r.uniform(-89, -86, E), r.normal(-100, 1, E), r.normal(-150, 30, E), r.uniform(30, 60, E),
                   r.uniform(-110, -90, E), r.uniform(-98, -85, E), r.normal(0, 40, E)]
    rows[-3][E // 3] = -20.0
    rows[-2][E // 2] = 0.0
    return np.stack(rows).astype(np.float32)


def check_choice(l, ids, k, score, bias, groups, top, group_score):
    """One token's ids: distinct, in order, and none left out that is better, to within TOL."""
    if bias is None and (top == groups or group_score == "max"):
        want = gate_ref.choose_token(l, k, score, None, groups, top, group_score)[0]
        np.testing.assert_array_equal(ids, want)
        return
    v = gate_ref.scores(l, score)[0] + (0 if bias is None else np.float64(bias))
    tol = TOL * max(1.0, 0 if bias is None else np.abs(bias).max())
    assert len(set(ids.tolist())) == k and (np.diff(v[ids]) <= 2 * tol).all()
    per = len(l) // groups
    best = -np.sort(-v.reshape(groups, per), axis=1)
    worth = best[:, 0] if group_score == "max" else best[:, :2].sum(1)
    border = np.sort(worth)[groups - top]
    assert (worth[ids // per] >= border - 4 * tol).all() and len(set((ids // per).tolist())) <= top
    sure = np.repeat(worth > border + 4 * tol, per) if top < groups else np.ones(len(l), bool)
    sure[ids] = False
    if sure.any():
        assert v[ids].min() >= v[sure].max() - 2 * tol


@pytest.mark.parametrize("T", [13, 9009])
@pytest.mark.parametrize("E,k,groups,top", [(64, 4, 1, 1), (256, 8, 8, 4), (160, 6, 8, 3), (512, 16, 16, 4)])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choice_and_weights(T, E, k, groups, top, with_bias, score):
    import torch

    from bit_mixture_experts_gb300 import _lib
    l = tokens(E, E + k)
    b = None
    if with_bias:
        b = (np.round(np.random.default_rng(E).standard_normal(E) * 40) * 0.001).astype(np.float32)
        b[E // 5] = 2.0  # an expert that is always chosen, whatever its score
    rows = np.arange(T) % len(l)
    for group_score, renorm in (("top2", True), ("max", True), ("top2", False)):
        gate = make(k, b, score=score, groups=groups, top_groups=top, group_score=group_score, renorm=renorm, scale=2.5)
        ids, w = (t.cpu().numpy() for t in gate.choose(torch.tensor(l[rows], device="cuda")))
        torch.cuda.synchronize()
        assert _lib.moe_get_device_error() == 0
        for t in range(len(l)):
            check_choice(l[t], ids[t], k, score, b, groups, top, group_score)
            want = gate_ref.weights(l[t], ids[t], score, renorm, 2.5)
            rel = REL
            if not renorm and score == "softmax":  # the sum over all (69 u, its terms 4 u and ln E u), the argument's rounding
                rel += (80 + np.abs(l[t].max() - l[t][ids[t]].astype(np.float64))) * 2.0 ** -24
            off = np.abs(w[t].astype(np.float64) - want) - (rel * want + 2.5 * 2.0 ** -126)
            assert (off <= 0).all(), (t, w[t], want)
        assert (ids == ids[rows]).all() and (w == w[rows]).all()


def test_the_weights_of_low_scores_by_hand():
    import torch
    # sigmoid(l) is e^l here: ratios 1 : e : 1/e
    for low in (-87.5, -88.0, -100.0, -1000.0):
        l = torch.full((1, 16), low - 5, device="cuda")
        l[0, :3] = torch.tensor([low, low + 1, low - 1], device="cuda")
        for bias in (None, np.zeros(16, np.float32)):
            ids, w = make(3, bias, score="sigmoid").choose(l)
            z = np.exp([0.0, 1.0, -1.0])[ids[0].cpu().numpy()]
            assert sorted(ids[0].tolist()) == [0, 1, 2]
            np.testing.assert_allclose(w[0].double().cpu().numpy(), z / z.sum(), rtol=REL)
    # softmax over the chosen: an expert that its bias alone brings in, 100 below the others
    l = torch.zeros((1, 16), device="cuda")
    l[0, 1] = -100.0
    b = np.zeros(16, np.float32)
    b[1] = 5.0
    ids, w = make(1, b, score="softmax").choose(l)
    assert ids.item() == 1 and w.item() == 1.0
