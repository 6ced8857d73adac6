"""Gates and residual norms in float64 (test infrastructure only): the definitions of include/moe_w4.h's moe_gate and
moe_residual_norm, a token at a time."""
from __future__ import annotations

import numpy as np


def scores(logits, score):
    """logits float [E] -> (scores float64 [E], those below 2^-126 as 0, which are available)."""
    l = np.asarray(logits, np.float64)
    here = l > -np.inf  # not NaN either
    l = np.where(here, np.minimum(l, np.finfo(np.float32).max), -np.inf)
    if not here.any():
        return np.zeros(len(l)), here
    with np.errstate(over="ignore"):
        if score == "softmax":
            e = np.exp(l - l.max())
            s = e / e.sum()
        else:
            s = 1.0 / (1.0 + np.exp(-l))
    return np.where(s < 2.0 ** -126, 0.0, s), here


def weights(logits, ids, score="softmax", renorm=True, scale=1.0):
    """The weights of one token's chosen experts: their scores' ratios (renorm), or the scores, those below 2^-126 as 0."""
    if not renorm:
        return scores(logits, score)[0][ids] * scale
    l = np.asarray(logits, np.float64)[ids]
    here = l > -np.inf
    if not here.any():
        return np.zeros(len(ids))
    l = np.minimum(l[here], np.finfo(np.float32).max)
    log_s = l if score == "softmax" else -np.logaddexp(0.0, -l)
    s = np.zeros(len(ids))
    s[here] = np.exp(log_s - log_s.max())
    return s / s.sum() * scale


def choose_token(logits, k, score="softmax", bias=None, groups=1, top_groups=None, group_score="top2", renorm=True,
                 scale=1.0):
    """One token's (ids int [k], weights float64 [k])."""
    E = len(logits)
    s, here = scores(logits, score)
    if bias is None and (group_score == "max" or top_groups in (None, groups)):
        v = np.asarray(logits, np.float64)  # scores are monotone in the logits
    else:
        v = s if bias is None else s + np.asarray(bias, np.float64)
    per = E // groups
    allowed = np.ones(E, bool)
    if top_groups is not None and top_groups < groups:
        worth = []
        for g in range(groups):
            best = sorted(v[g * per:(g + 1) * per][here[g * per:(g + 1) * per]], reverse=True)
            worth.append(-np.inf if not best else best[0] if group_score == "max" else sum(best[:2]))
        stay = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
        allowed = np.isin(np.arange(E) // per, stay)
    order = sorted((e for e in range(E) if allowed[e]), key=lambda e: (not here[e], -v[e] if here[e] else 0.0, e))
    ids = np.array(order[:k])
    return ids, weights(logits, ids, score, renorm, scale)


def choose(logits, k, **kw):
    """logits [T, E] -> (ids int32 [T, k], weights float64 [T, k])."""
    both = [choose_token(row, k, **kw) for row in np.asarray(logits)]
    if not both:
        return np.zeros((0, k), np.int32), np.zeros((0, k))
    return np.stack([b[0] for b in both]).astype(np.int32), np.stack([b[1] for b in both])


def choose_many(logits, k, score="softmax", bias=None, groups=1, top_groups=None, group_score="top2", renorm=True,
                scale=1.0):
    """choose for many tokens at a time, all of whose logits are finite."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    if score == "softmax":
        s = np.exp(l - l.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    else:
        s = 1.0 / (1.0 + np.exp(-l))
    dropping = top_groups is not None and top_groups < groups
    v = s + np.asarray(bias, np.float64) if bias is not None else s if dropping and group_score == "top2" else l
    if dropping:
        best = -np.sort(-v.reshape(T, groups, -1), axis=2)
        worth = best[:, :, 0] if group_score == "max" else best[:, :, :2].sum(2)
        stay = np.argsort(-worth, axis=1, kind="stable")[:, :top_groups]
        allowed = np.zeros((T, groups), bool)
        np.put_along_axis(allowed, stay, True, 1)
        v = np.where(np.repeat(allowed, E // groups, 1), v, -np.inf)
    ids = np.argsort(-v, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(s, ids, 1)
    return ids.astype(np.int32), (w / w.sum(1, keepdims=True) if renorm else w) * scale


def sort_assignments(ids, E):
    """ids [T, k] -> (counts, offsets, perm, inv_perm) of moe_route."""
    flat = np.asarray(ids).reshape(-1)
    perm = np.array(sorted(range(len(flat)), key=lambda a: (flat[a], a)), np.int32)
    inv = np.empty_like(perm)
    inv[perm] = np.arange(len(flat))
    counts = np.bincount(flat, minlength=E).astype(np.int32)
    return counts, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), perm, inv


def combined(y, inv_perm, topk_w):
    """Each token's weighted sum of its rows of y and its shared row; also the sum of the terms' sizes."""
    T, k = topk_w.shape
    y, w = np.asarray(y, np.float64), np.asarray(topk_w, np.float64)
    rows = y[np.asarray(inv_perm).reshape(T, k)]
    shared = y[T * k:]
    return (w[:, :, None] * rows).sum(1) + shared, (np.abs(w)[:, :, None] * np.abs(rows)).sum(1) + np.abs(shared)


def residual(x, y, w_pre=None, w_post=None, gate=None, scale=1.0, eps=1e-6, offset=0.0, post=None, y_size=None, terms=0,
             depth=80):
    """(r, n, bound of r's error, bound of n's error) in float64, the bounds for FP32 arithmetic before the outputs'
    rounding.  y None: r = scale x.  `y_size`, `terms`: y is itself an FP32 sum of that many terms whose sizes add up to
    y_size.  `depth`: additions on a value's way into a row's sum of squares.

    In units of u = 2^-24: a sum of squares is off by (depth + 1) u, its root by half of that, the mean's division, eps,
    the root and the reciprocal by one each, every product and sum behind it by one."""
    u = 2.0 ** -24
    x = np.asarray(x, np.float64) * scale
    norm = (depth + 1) / 2 * u + 4 * u
    if y is None:
        r, dr = x, 2 * u * np.abs(x)
    else:
        z = np.asarray(y, np.float64)
        dz = np.zeros_like(z) if y_size is None else (terms + 1) * u * y_size
        if post if post is not None else w_post is not None:
            g = np.ones(z.shape[1]) if w_post is None else np.asarray(w_post, np.float64) + offset
            rms = np.sqrt((z * z).mean(1, keepdims=True) + eps)
            off = np.sqrt((dz * dz).mean(1, keepdims=True)) / rms + norm
            z, dz = z / rms * g, np.abs(g) / rms * dz
            dz = dz + np.abs(z) * (off + 3 * u)
        if gate is not None:
            g = np.asarray(gate, np.float64)
            z, dz = z * g, dz * np.abs(g)
            dz = dz + u * np.abs(z)
        r = x + z
        dr = dz + 2 * u * (np.abs(x) + np.abs(z))
    g = np.ones(r.shape[1]) if w_pre is None else np.asarray(w_pre, np.float64) + offset
    rms = np.sqrt((r * r).mean(1, keepdims=True) + eps)
    off = np.sqrt((dr * dr).mean(1, keepdims=True)) / rms + norm
    n = r / rms * g
    return r, n, dr, np.abs(g) / rms * dr + np.abs(n) * (off + 3 * u)
