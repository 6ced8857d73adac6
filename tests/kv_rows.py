"""Chosen rows of a large attention call against the float64 oracle, with the error bounds of tests/kv_util.py
for each row."""
from __future__ import annotations

import numpy as np

from oracle import kv_ref


def check_rows(s, out, lse, rows, scale=None, chain=None, what=""):
    """Rows `rows` (of T) of a call on the batch of kv_util.Setup `s`.  `chain`: how many FP32 additions in a row
    a sum over all keys takes at most, by the number of keys (each key one addition, unless given)."""
    scale = s.d ** -0.5 if scale is None else scale
    pools, q = s.values(), s.q.double().cpu().numpy()
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    cached = {}
    for i in rows:
        b = int(np.searchsorted(s.cu, i, side="right")) - 1
        if b not in cached:
            cached = {b: [kv_ref.gather(x, s.table[b], s.kv_lens[b]) for x in pools]}
        p = s.kv_lens[b] - s.q_lens[b] + int(i) - int(s.cu[b])
        ref, ref_lse, mag, smag = kv_ref.attention(q[i:i + 1], *(x[:p + 1] for x in cached[b]), 1, scale)
        n = (p + 1 if chain is None else chain(p + 1)) * 2.0 ** -24
        # as in kv_util.Setup.reference: the scores' error, then the weights', the sums' and the output's
        ds = smag * (2.0 ** -20 * np.sqrt(s.d / 16 + 8) + 2.0 ** -22) + 2.0 ** -22
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * ds + 2 * n)[..., None] * mag * 1.01 + 1e-30
        tol_lse = ds + n + 2.0 ** -21 * (1 + np.abs(ref_lse))
        bad = ~(np.abs(got[i] - ref[0]) <= tol[0])
        assert not bad.any(), (f"{what} row {i} (position {p}): {bad.sum()} of {bad.size} outputs outside their bound, got "
                               f"{got[i][bad][0]}, exact {ref[0][bad][0]}, bound {tol[0][bad][0]}")
        bad = ~(np.abs(got_lse[i] - ref_lse[0]) <= tol_lse[0])
        assert not bad.any(), f"{what} row {i} (position {p}): log-sum-exp {got_lse[i][bad]}, exact {ref_lse[0][bad]}"


def spread(lo, hi, n):
    """About n rows of lo .. hi - 1, the first and the last among them, none in step with a tile."""
    r = np.random.default_rng(hi)
    return np.unique(np.concatenate([[lo, hi - 1], r.integers(lo, hi, n)]))
