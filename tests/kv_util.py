"""Helpers of the paged key/value cache tests: batches with shuffled pages whose unused rows hold NaN, and the
error bounds of the attention."""
from __future__ import annotations

import numpy as np

from oracle import kv_ref


class Setup:
    """A cache (GPU) with its pages handed out in random order, holding random values for every sequence's
    kv_len tokens and NaN everywhere else (pages of nobody, rows past kv_len, their scales)."""

    def __init__(self, q_lens, kv_lens, heads=2, g=4, d=128, page=16, fmt="bf16", seed=0, extra_width=1, sigma=1.0):
        import torch
        from bit_mixture_experts_gb300 import PagedKVCache
        self.q_lens, self.kv_lens, self.heads, self.hq, self.d, self.page, self.fmt = (
            list(q_lens), list(kv_lens), heads, heads * g, d, page, fmt)
        self.dev = dev = torch.device("cuda:0")
        r = self.rng = np.random.default_rng(seed)
        need = [-(-c // page) for c in kv_lens]
        n_pages = sum(need) + 2
        order = r.permutation(n_pages).astype(np.int32)
        self.table = np.full((len(kv_lens), max(need) + extra_width), -1, np.int32)  # unused entries: no page
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.T = sum(q_lens)
        self.cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        shape = (n_pages, heads, page, d)
        live = np.zeros((n_pages, page), bool)
        for b, c in enumerate(kv_lens):
            for p in range(c):
                live[self.table[b, p // page], p % page] = True
        pools = []
        for _ in range(2):
            x = torch.from_numpy(r.standard_normal(shape).astype(np.float32) * sigma).bfloat16()
            keep = torch.from_numpy(live)[:, None, :].expand(n_pages, heads, page)
            if fmt == "bf16":
                x[~keep] = float("nan")
                pools += [x.to(dev), None]
            else:
                codes, s = kv_ref.quantise(x.double().numpy())
                s = torch.from_numpy(s.astype(np.float32))
                codes = torch.from_numpy(codes)
                codes[~keep] = 0x7f
                s[~keep] = float("nan")
                pools += [codes.view(torch.float8_e4m3fn).to(dev), s.to(dev)]
        k, ks, v, vs = pools
        self.cache = PagedKVCache.from_tensors(k, v, ks, vs)
        self.idx = [torch.from_numpy(a).to(dev) for a in (self.table, self.cu, np.asarray(kv_lens, np.int32))]
        self.batch = self.cache.batch(*self.idx, self.T)
        self.q = torch.from_numpy(r.standard_normal((self.T, self.hq, d)).astype(np.float32)).bfloat16().to(dev)

    def values(self):
        """The pools' values in float64."""
        out = []
        for x, s in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            y = x.float().double().cpu().numpy()
            out.append(y if s is None else y * s.double().cpu().numpy()[..., None])
        return out

    def reference(self, scale=None, q=None):
        """(out, lse, tol_out, tol_lse) of the attention over all rows of T."""
        scale = self.d ** -0.5 if scale is None else scale
        k, v = self.values()
        q = (self.q if q is None else q).double().cpu().numpy()
        parts = []
        for b, (n, c) in enumerate(zip(self.q_lens, self.kv_lens)):
            kk, vv = (kv_ref.gather(x, self.table[b], c) for x in (k, v))
            parts.append(kv_ref.attention(q[self.cu[b]:self.cu[b + 1]], kk, vv, n, scale))
        out, lse, mag, smag = (np.concatenate([p[i] for p in parts]) for i in range(4))
        # Scores: bf16 products summed in FP32 in some order, d/16 partial sums of 16: relative to the sum of
        # magnitudes at most 2^-20 sqrt(d / 16 + 8) as for the router's logits (tests/test_route_x_gpu.py);
        # plus the rounding of scale * log2(e) and of the exponent's argument, 2^-22 of the scores' size.
        ds = smag * (2.0 ** -20 * np.sqrt(self.d / 16 + 8) + 2.0 ** -22) + 2.0 ** -22
        # Weights: exp's error ds on top and bottom (2 ds), rounded to bf16 (half an ulp, 2^-8 at most) for the
        # product; sums of n weights in FP32, at most n 2^-24; the output rounded to bf16 once.
        n = max(self.kv_lens) if self.kv_lens else 1
        tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * ds + 2 * n * 2.0 ** -24)[..., None] * mag * 1.01 + 1e-30
        with np.errstate(invalid="ignore"):
            tol_lse = ds + n * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))
        return out, lse, tol, tol_lse


def check(setup, out, lse=None, what="", **kw):
    ref, ref_lse, tol, tol_lse = setup.reference(**kw)
    got = out.double().cpu().numpy()
    assert got.shape == ref.shape
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outputs outside their bound, first at "
                           f"{tuple(np.argwhere(bad)[0])}: got {got[bad][0]}, exact {ref[bad][0]}, bound {tol[bad][0]}")
    if lse is not None:
        g = lse.double().cpu().numpy()
        empty = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(g), empty), what
        assert np.all(np.abs(g[~empty] - ref_lse[~empty]) <= tol_lse[~empty]), what
