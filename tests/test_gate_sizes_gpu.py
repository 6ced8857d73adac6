"""Numbers of experts that leave lanes of a warp without any although the others have eight each, whole and with many
experts that are not available: none of another group's or beyond the last is ever named."""
import numpy as np
import pytest

from test_gate_gpu import check, draw

pytestmark = pytest.mark.gpu


def setup_module():
    import gpu_util
    gpu_util.ensure_built()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E,groups,top", [(232, 1, 1), (240, 1, 1), (248, 1, 1), (240, 2, 1), (240, 2, 2), (256, 2, 1), (256, 4, 3)])
@pytest.mark.parametrize("k", [8, 32])
def test_lanes_without_experts(E, groups, top, k, with_bias, score):
    l, b = draw(40, E, E + k)
    r = np.random.default_rng(E)
    l[5] = -np.inf
    l[6, 3:] = np.nan
    l[7, :E // 2] = -np.inf           # all of the first group, where there are two
    l[8, E // 2 + 1:] = -np.inf       # all but one of the second
    for t in range(9, 25):
        l[t, r.permutation(E)[:E - 1 - t]] = -np.inf  # fewer left than are chosen
    for how in ("top2", "max"):
        check(l, k, b if with_bias else None, score=score, groups=groups, top_groups=top, group_score=how, scale=1.5)
