"""Float64 restatement of the paged key/value cache operators (append, read, attention).

Sequences are given as Python lists; pages as NumPy arrays [num_pages, heads, page_size, d].  e4m3 codes are
decoded and rounded by way of a table of all values of the format, built from its definition (1 sign bit, 4
exponent bits with bias 7, 3 fraction bits, subnormals, no infinities, code 127 NaN).
"""
from __future__ import annotations

import numpy as np


def e4m3_table() -> np.ndarray:
    """Value of every code 0..255 in float64 (NaN at 127 and 255)."""
    out = np.empty(256)
    for c in range(128):
        e, m = c >> 3, c & 7
        out[c] = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    out[127] = np.nan
    out[128:] = -out[:128]
    return out


TABLE = e4m3_table()


def e4m3_codes(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code of each float64 |x| <= 448 (ties to the even code, sign kept)."""
    mag = TABLE[:127]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(mag, a), 1, 126)
    lo = hi - 1
    d_lo, d_hi = a - mag[lo], mag[hi] - a
    pick = np.where(d_lo < d_hi, lo, np.where(d_hi < d_lo, hi, np.where(lo % 2 == 0, lo, hi)))
    return (pick + 128 * np.signbit(x)).astype(np.uint8)


def row_scale(x: np.ndarray) -> np.ndarray:
    """Per row (last axis): the least power of two 2^e, e >= -126, with max|x| <= 448 * 2^e; 1 for zeros."""
    a = np.abs(x).max(-1)
    out = np.ones_like(a)
    for i, v in np.ndenumerate(a):
        if v > 0:
            e = -126
            while v > 448.0 * 2.0 ** e:
                e += 1
            out[i] = 2.0 ** e
    return out


def quantise(x: np.ndarray):
    """float64 rows [..., d] -> (codes uint8, scale float64 [...])."""
    s = row_scale(x)
    return e4m3_codes(x / s[..., None]), s


def positions(n: int, kv_len: int) -> list:
    """Positions of a sequence's n new tokens (negative ones exist in no page)."""
    return [kv_len - n + i for i in range(n)]


def gather(pages: np.ndarray, table_row, kv_len: int) -> np.ndarray:
    """A sequence's cached rows in order, [kv_len, heads, d]."""
    P = pages.shape[2]
    if kv_len == 0:
        return np.zeros((0, pages.shape[1], pages.shape[3]))
    return np.stack([pages[table_row[p // P], :, p % P] for p in range(kv_len)])


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, n: int, scale: float):
    """One sequence: q [n, q_heads, d] over k, v [kv_len, heads, d], all float64.  Returns the output, the
    log-sum-exp, sum_j w_j |v_j| / sum_j w_j (the scale of the output's rounding errors) and
    max_j scale * sum_c |q_c k_jc| per (token, head) (that of the scores')."""
    L, heads, d = k.shape
    hq = q.shape[1]
    out, mag = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse, smag = np.full((n, hq), -np.inf), np.zeros((n, hq))
    for i, p in enumerate(positions(n, L)):
        if p < 0:
            continue
        for h in range(hq):
            kk, vv = k[:p + 1, h * heads // hq], v[:p + 1, h * heads // hq]
            s = scale * (kk @ q[i, h])
            m = s.max()
            w = np.exp(s - m)
            out[i, h] = w @ vv / w.sum()
            mag[i, h] = w @ np.abs(vv) / w.sum()
            lse[i, h] = m + np.log(w.sum())
            smag[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, lse, mag, smag
