"""A decoder block over the paged key/value cache: attention, then the W4 mixture-of-experts layer.

    python -m bit_mixture_experts_gb300.block [--fmt e4m3] [--prompts 300,45] [--chunk 128] [--steps 8] [--gated]

The command serves a ragged batch as a server would: the prompts go through the block in chunks, all
sequences' chunks of a step packed into one batch; then one token per sequence and step.  It needs a GPU and
is run from the repository root (the synthetic weights come from `workloads`).  PyTorch does the block's two
dense bf16 projections and, in a block without `norms`, the residual additions; norms, cache, attention,
router and experts are libmoe_w4.so's kernels.  There is no positional encoding.  With --gated the experts are
chosen by sigmoid scores with a bias in groups, and the block has norms with gains before and after its
attention and its experts, a gate per channel and a residual stream in 32 bits.
"""
from __future__ import annotations

import argparse

from . import _lib
from .gate import ExpertGate
from .kv import PagedKVCache
from .layer import MoELayerW4, _dev
from .residual import ResidualNorm


class DecoderBlockW4:
    """x + attention(norm(x)) W_o, then that plus the experts of its own norm.

    w_qkv is bf16 [(q_heads + 2 * cache.heads) * d, H] (all query heads, then keys, then values), w_o bf16
    [H, q_heads * d], w_router bf16 [E, H], `moe` a MoELayerW4 and `cache` a PagedKVCache.

    `norms`: three ResidualNorm for a block with gains, post-norms, gates and scales of its own: of the block's input,
    around the addition of the attention's output (its n is what router and experts take), and around that of the
    experts' (its n is what the next block's attention takes).  `gates`: their gates' values per channel, or None.
    Such a block's router is moe_router at every size: E a multiple of 64, at most 512.
    """

    def __init__(self, w_qkv, w_o, w_router, moe: MoELayerW4, cache: PagedKVCache, norms=None, gates=(None, None)):
        self.q_heads = w_o.shape[1] // cache.d
        want = ((self.q_heads + 2 * cache.heads) * cache.d, moe.H)
        if tuple(w_qkv.shape) != want or w_o.shape[0] != moe.H or tuple(w_router.shape) != (moe.E, moe.H):
            raise ValueError(f"w_qkv must be {want}, w_o [{moe.H}, q_heads * {cache.d}], w_router "
                             f"[{moe.E}, {moe.H}]: got {tuple(w_qkv.shape)}, {tuple(w_o.shape)}, "
                             f"{tuple(w_router.shape)}")
        if w_o.shape[1] % cache.d or self.q_heads % cache.heads:
            raise ValueError(f"w_o's {w_o.shape[1]} columns must be q_heads * {cache.d}, q_heads a multiple of the cache's "
                             f"{cache.heads} heads")
        if norms is not None and len(norms) != 3:
            raise ValueError(f"three norms are needed, got {len(norms)}")
        self.norms, self.gates = norms, gates
        self.w_qkv, self.w_o, self.w_router, self.moe, self.cache = w_qkv, w_o, w_router, moe, cache

    def project(self, x, xn=None):
        """Queries, keys and values of the normed x (xn, if it is known): slices of one [T, q_heads + 2 heads, d]
        tensor, which the cache and the attention read where they are."""
        import torch
        if xn is None:
            xn = torch.empty_like(x)
            _lib.moe_rms_norm(x, xn)
        hq, hkv = self.q_heads, self.cache.heads
        return (xn @ self.w_qkv.T).view(x.shape[0], hq + 2 * hkv, self.cache.d).split((hq, hkv, hkv), dim=1)

    def attend(self, x, batch, xn=None):
        """The new tokens' attention output, bf16 [T, q_heads, d]; their keys and values enter the cache."""
        q, k, v = self.project(x, xn)
        self.cache.append(k, v, batch)
        return self.cache.attention(q, batch)

    def experts(self, x):
        """The W4 experts of the normed x, bf16 [T, H]."""
        import torch
        T, (E, k) = x.shape[0], (self.moe.E, self.moe.k)
        xn = torch.empty_like(x)
        logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
        if T <= 8:  # the decode step's launch for both
            _lib.moe_norm_router(x, self.w_router, xn, logits)
        else:
            _lib.moe_rms_norm(x, xn)
            ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
            w = torch.empty((T, k), dtype=torch.float32, device=x.device)
            _lib.moe_router(xn, self.w_router, k, logits, ids, w)
        return self.moe.forward(xn, logits)

    def forward(self, x, batch):
        """x bf16 [T, H], the new tokens of `batch`'s sequences (cache.batch) -> bf16 [T, H].  With `norms` the residual
        stream may also be float32; the result then is too."""
        if self.norms is not None:
            return self.forward_stream(x, self.norms[0].norm(x), batch)[0]
        x = x + self.attend(x, batch).view(x.shape[0], -1) @ self.w_o.T
        return x + self.experts(x)

    def forward_stream(self, x, xn, batch):
        """One block of a stack with `norms`: the residual stream x (bf16 or float32 [T, H]) and its norm xn (bf16) ->
        both after the block; the next block's forward_stream takes them."""
        import torch
        T, E, k = x.shape[0], self.moe.E, self.moe.k
        _, around_attention, around_experts = self.norms
        y = self.attend(x, batch, xn).view(T, -1) @ self.w_o.T
        x, xn = around_attention.add(x, y, self.gates[0])
        logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
        ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
        _lib.moe_router(xn, self.w_router, k, logits, ids, torch.empty((T, k), dtype=torch.float32, device=x.device))
        return self.moe.forward_residual(xn, logits, x, around_experts, self.gates[1])


def synthetic(shape, q_heads=16, kv_heads=2, d=128, fmt="bf16", num_pages=256, page_size=64, seed=0, device="cuda",
              gated=False):
    """A block of random weights: experts and router from `workloads`, projections of unit-variance outputs; `gated`:
    with a gate of sigmoid scores, a bias and groups, and with norms."""
    import torch

    import workloads
    gen = torch.Generator().manual_seed(seed)

    def dense(rows, cols):
        return (torch.randn((rows, cols), generator=gen) * cols ** -0.5).bfloat16().to(device)

    gate = norms = None
    gates = (None, None)
    if gated:
        def gains():
            return (1 + 0.2 * torch.randn(shape.H, generator=gen)).to(device)

        bias = (torch.randn(shape.E, generator=gen) * 20).round().mul(0.001).to(device)
        groups = 4 if shape.E % 4 == 0 else 1
        gate = ExpertGate(shape.k, "sigmoid", bias, groups, max(1, groups // 2), scale=2.5)
        norms = ResidualNorm(gains()), ResidualNorm(gains(), gains()), ResidualNorm(gains(), gains(), scale=0.9)
        gates = 0.5 * gains(), 0.5 * gains()
    moe = MoELayerW4(shape.H, shape.E, shape.k, shape.F, workloads.make_weights(shape, seed), device=device, gate=gate)
    router = _dev(workloads.router_weight_bits(shape, seed), device).view(torch.bfloat16)
    cache = PagedKVCache(num_pages, page_size, kv_heads, d, fmt, device)
    return DecoderBlockW4(dense((q_heads + 2 * kv_heads) * d, shape.H), dense(shape.H, q_heads * d), router, moe, cache,
                          norms, gates)


def serve(block, prompts, chunk, steps):
    """Runs `prompts` (one bf16 [n, H] each) in chunks of up to `chunk` tokens per sequence, then `steps`
    steps of one token per sequence, the block's last output of each sequence being its next input.  Yields
    (x, new tokens per sequence, kv_len, page table, output) of every step.  Every prompt has a token: its
    output is what the next steps go on from."""
    import torch
    if not prompts or not all(len(p) for p in prompts):
        raise ValueError(f"prompts of at least one token are needed, got lengths {[len(p) for p in prompts]}")
    if chunk < 1 or steps < 0:
        raise ValueError(f"chunk {chunk} must be at least 1 and steps {steps} not negative")
    cache, dev = block.cache, prompts[0].device
    need = [-(-(len(p) + steps) // cache.page_size) for p in prompts]
    if sum(need) > cache.num_pages:
        raise ValueError(f"{sum(need)} pages needed, the cache has {cache.num_pages}")
    table = torch.zeros((len(prompts), max(need)), dtype=torch.int32)
    pages = torch.randperm(cache.num_pages).int()  # handed out in no order, as after some hours of service
    for b, n in enumerate(need):
        table[b, :n] = pages[sum(need[:b]):sum(need[:b + 1])]
    table = table.to(dev)
    done = [0] * len(prompts)
    last = [None] * len(prompts)
    while True:
        new = [p[at:at + chunk] for p, at in zip(prompts, done)]
        if not any(len(n) for n in new):  # all prompts are in
            if steps == 0:
                return
            steps -= 1
            new = last
        n_new = [len(n) for n in new]
        done = [at + n for at, n in zip(done, n_new)]
        cu = torch.tensor([sum(n_new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device=dev)
        kv_len = torch.tensor(done, dtype=torch.int32, device=dev)
        x = torch.cat(new)
        out = block.forward(x, cache.batch(table, cu, kv_len, len(x)))
        for b, o in enumerate(out.split(n_new)):
            if len(o):
                last[b] = o[-1:]
        yield x, n_new, done, table, out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n", 1)[0])
    ap.add_argument("--fmt", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--prompts", default="300,45", help="prompt lengths, comma-separated")
    ap.add_argument("--chunk", type=int, default=128)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--gated", action="store_true", help="a gate and norms with gains (see above)")
    args = ap.parse_args(argv)
    import torch

    import workloads
    block = synthetic(workloads.FULL, fmt=args.fmt, gated=args.gated)
    gen = torch.Generator().manual_seed(1)
    stream = torch.float32 if args.gated else torch.bfloat16
    prompts = [torch.randn((int(n), workloads.FULL.H), generator=gen).to(stream).cuda() for n in args.prompts.split(",")]
    for i, (x, new, lens, _, out) in enumerate(serve(block, prompts, args.chunk, args.steps)):
        torch.cuda.synchronize()
        err = _lib.moe_get_device_error()
        if err:
            raise SystemExit(f"step {i}: device error {err}")
        print(f"step {i}: {len(x)} new tokens {new}, cached {list(lens)}, output rms {out.float().square().mean().sqrt():.4f}")


if __name__ == "__main__":
    main()
