"""Value rows of which a few elements alone are infinite or NaN: those elements' columns carry them to the
tokens that see the key, every other column keeps what the row's finite elements give (checked column by
column against the float64 oracle, in every form of the attention)."""
import numpy as np
import pytest

import gpu_util as G
import kv_util as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _pair_tokens(heads, tpt):
    """Tokens of one sequence whose query tiles go in pairs: more than one pair for every two SMs."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return 2 * tpt * (sms // (2 * heads) + 1)


# new tokens (None: as many as make pairs), tokens before them, KV heads, query heads per KV head
FORMS = {"rows to 8": (2, 300, 2, 4), "rows to 16": (4, 300, 2, 4), "rows to 32": (8, 300, 2, 4),
         "rows to 32, cut": (5, 3000, 1, 5), "tile": (40, 100, 2, 4), "tiles, cut": (70, 3000, 1, 8),
         "prompt": (200, 0, 2, 2), "pairs": (None, 50, 8, 16)}


@pytest.mark.parametrize("d,page", [(64, 16), (128, 48)])
@pytest.mark.parametrize("form", list(FORMS))
def test_value_rows_with_some_elements_not_finite(form, d, page):
    import torch
    new, past, heads, g = FORMS[form]
    new = new or _pair_tokens(heads, 128 // g)
    n = new + past
    s = K.Setup([new], [n], heads=heads, g=g, d=d, page=page, seed=len(form))
    r = np.random.default_rng(d)
    # new tokens' rows (not the first one's alone: tokens that do not see a row must stay as they are), and
    # one that all tokens see
    at = sorted({n - 1, n - new // 2 - 1, past + min(1, new - 1)} | ({past // 2} if past else set()))
    for i, p in enumerate(at):
        h, cols = i % heads, r.choice(d, 3, replace=False)
        for c, x in zip(cols[:1 + i % 3], (np.inf, -np.inf, np.nan)):
            s.cache.v[int(s.table[0, p // page]), h, p % page, int(c)] = x
    out, lse = s.cache.attention(s.q, s.batch, return_lse=True)
    torch.cuda.synchronize()
    from bit_mixture_experts_gb300 import _lib
    assert _lib.moe_get_device_error() == 0
    with np.errstate(invalid="ignore"):
        ref, ref_lse, tol, tol_lse = s.reference()
    got, fin = out.double().cpu().numpy(), np.isfinite(ref)
    assert not fin.all() and fin.any(-1).all()
    bad = ~(np.abs(got[fin] - ref[fin]) <= tol[fin])
    assert not bad.any(), (f"{bad.sum()} of {bad.size} finite outputs outside their bound: got {got[fin][bad][:4]}, "
                           f"exact {ref[fin][bad][:4]}")
    assert np.array_equal(got[~fin], ref[~fin], equal_nan=True)
    assert np.all(np.abs(lse.double().cpu().numpy() - ref_lse) <= tol_lse)
