"""A decoder block served in chunks and then token by token (bit_mixture_experts_gb300/block.py): at every step
the attention of the block against the float64 oracle over all keys and values that the block has projected so
far, and the block's output against its parts.  The prompts are ragged, one runs out of chunks before the
other, and the cache's pages are handed out in random order."""
import numpy as np
import pytest

import workloads
from oracle import kv_ref

import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_block_in_chunks_then_token_by_token(fmt):
    import torch
    from bit_mixture_experts_gb300 import _lib, block
    shape, d, scale = workloads.LayerShape(H=256, E=64, k=4, F=128), 64, 64 ** -0.5
    blk = block.synthetic(shape, q_heads=8, kv_heads=2, d=d, fmt=fmt, num_pages=24, page_size=16, device=G.torch_dev())
    attended = []
    attend = blk.attend

    def recording(x, batch):
        attended.append(attend(x, batch))
        return attended[-1]

    blk.attend = recording
    gen = torch.Generator().manual_seed(3)
    lens = (75, 9, 1)
    prompts = [torch.randn((n, shape.H), generator=gen).bfloat16().to(G.torch_dev()) for n in lens]
    ks, vs = [[] for _ in lens], [[] for _ in lens]
    kinds = set()
    for step, (x, new, kv_len, _, out) in enumerate(block.serve(blk, prompts, 32, 5)):
        torch.cuda.synchronize()
        assert _lib.moe_get_device_error() == 0
        q, k, v = (_f64(t) for t in blk.project(x))  # the same call on the same input: the same bits
        if fmt == "e4m3":
            k, v = (kv_ref.TABLE[c] * s[..., None] for c, s in (kv_ref.quantise(k), kv_ref.quantise(v)))
        o = attended[step]
        at = 0
        for b, n in enumerate(new):
            rows = slice(at, at + n)
            at += n
            ks[b].append(k[rows])
            vs[b].append(v[rows])
            kk, vv = np.concatenate(ks[b]), np.concatenate(vs[b])
            assert len(kk) == kv_len[b]
            if n == 0:
                continue
            kinds.add("decode" if n == 1 else "chunk")
            exact, _, mag, smag = kv_ref.attention(q[rows], kk, vv, n, scale)
            # the bound of the attention's roundings (tests/kv_util.py)
            ds = smag * (2.0 ** -20 * np.sqrt(d / 16 + 8) + 2.0 ** -22) + 2.0 ** -22
            tol = 2.0 ** -8 * np.abs(exact) + (2.0 ** -8 + 2 * ds + 2 * len(kk) * 2.0 ** -24)[..., None] * mag * 1.01
            assert np.all(np.abs(_f64(o[rows]) - exact) <= tol + 1e-30), f"step {step} sequence {b}"
        y = x + o.view(len(x), -1) @ blk.w_o.T
        assert torch.equal(out, y + blk.experts(y)), f"step {step}"
        assert torch.isfinite(out).all()
    assert kinds == {"decode", "chunk"} and step == 7  # chunks of 32, 32 and 11, then five tokens each


def test_block_refuses_weights_of_other_sizes():
    from bit_mixture_experts_gb300 import block
    blk = block.synthetic(workloads.TINY, q_heads=8, kv_heads=2, d=64, num_pages=4, page_size=16, device=G.torch_dev())
    with pytest.raises(ValueError, match="w_qkv"):
        block.DecoderBlockW4(blk.w_qkv[1:], blk.w_o, blk.w_router, blk.moe, blk.cache)
    with pytest.raises(ValueError, match="pages"):
        next(block.serve(blk, [blk.w_router] * 8, 32, 0))
