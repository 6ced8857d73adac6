"""The layer with a gate and with the residual addition that follows it, in every form of its kernels, and the decoder
block that runs them together: attention, norms, router, gate, experts, combine."""
import numpy as np
import pytest

import gpu_util as G
import workloads
from oracle import gate_ref
from test_residual_gpu import STEP, check_rows, f64

pytestmark = pytest.mark.gpu

KW = dict(score="sigmoid", groups=4, top_groups=2, scale=2.5)


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def bias_of(E, seed=0):
    import torch
    return (torch.randn(E, generator=torch.Generator().manual_seed(seed)) * 30).round().mul(0.001).cuda()


def make(T, impl="auto", gate=None, H=256, E=64, k=4, F=256, seed=0):
    from bit_mixture_experts_gb300.layer import MoELayerW4
    d = G.workload((T, H, E, k, F, False), seed)
    return (d, MoELayerW4(H, E, k, F, d, device=G.torch_dev(), impl=impl, gate=gate)) + G.to_dev_inputs(d)


def no_error():
    import torch

    from bit_mixture_experts_gb300 import _lib
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 0


def expected(layer, T, residual, norm, gate=None):
    """r and n of the rows of y that the layer's last call left, with their bounds."""
    b = layer.buffers(T)
    y, size = gate_ref.combined(f64(b["y"]), b["inv_perm"].cpu().numpy(), f64(b["topk_w"]))
    return gate_ref.residual(f64(residual), y, f64(norm.w_pre), f64(norm.w_post), f64(gate), norm.scale, norm.eps,
                             norm.offset, y_size=size, terms=layer.k + 1)


@pytest.mark.parametrize("T,impl", [(1, "auto"), (8, "auto"), (3, "tc"), (12, "gemv"), (64, "auto"), (600, "auto"),
                                    (2000, "tc"), (200, "tc_bf16")])
def test_the_default_gate_is_the_layer_without_one(T, impl):
    import torch

    from bit_mixture_experts_gb300 import ExpertGate
    d, plain, x, logits = make(T, impl)
    _, gated, _, _ = make(T, impl, ExpertGate(4))
    a, b = plain.forward(x, logits), gated.forward(x, logits)
    no_error()
    assert torch.equal(a, b)
    for name in ("topk_ids", "topk_w", "counts", "offsets", "perm", "inv_perm", "num_blocks"):
        assert torch.equal(plain.buffers(T)[name], gated.buffers(T)[name]), name


@pytest.mark.parametrize("T,impl", [(1, "auto"), (5, "auto"), (8, "tc"), (16, "gemv"), (77, "auto"), (1500, "auto")])
def test_a_gate_and_what_follows_the_layer(T, impl):
    import torch

    from bit_mixture_experts_gb300 import ExpertGate, ResidualNorm, _lib
    gate = ExpertGate(4, bias=bias_of(64), **KW)
    d, layer, x, logits = make(T, impl, gate)
    out = layer.forward(x, logits)
    no_error()
    b = layer.buffers(T)
    ids, w = gate.choose(logits)
    assert torch.equal(ids, b["topk_ids"]) and torch.equal(w, b["topk_w"])
    y = b["y"].clone()
    again = torch.empty_like(out)
    _lib.moe_combine(b["y"], b["inv_perm"], b["topk_w"], again)
    assert torch.equal(out, again)
    # the rows of y are those of the layer without a gate for logits with the same order: the same bits
    order = torch.full((T, 64), -50.0, device="cuda").scatter_(1, ids.long(), torch.arange(4, 0, -1.0, device="cuda").expand(T, 4))
    _, plain, _, _ = make(T, impl)
    plain.forward(x, order)
    no_error()
    assert torch.equal(plain.buffers(T)["topk_ids"], ids)
    assert torch.equal(plain.buffers(T)["y"], y)
    # with what follows: in every type, by logits and by a choice made before, r in the stream's place
    for stream, post in ((torch.bfloat16, True), (torch.float32, False)):
        gen = torch.Generator(device="cuda").manual_seed(T)
        res = torch.randn((T, 256), generator=gen, device="cuda").to(stream)
        gains = [torch.rand(256, generator=gen, device="cuda") + 0.5 for _ in range(3)]
        norm = ResidualNorm(gains[0], gains[1] if post else None, scale=0.9)
        want = None
        for how in (dict(logits=logits), dict(logits=None, choice=(ids, w))):
            b["y"].fill_(float("nan"))
            r, n = layer.forward_residual(x, residual=res, norm=norm, gate=gains[2], **how)
            no_error()
            assert torch.equal(b["y"], y)
            if want is None:
                want = expected(layer, T, res, norm, gains[2])
                check_rows(r, want[0], want[2], STEP["bf16" if stream == torch.bfloat16 else "f32"], "r")
                check_rows(n, want[1], want[3], STEP["bf16"], "n")
                first = r, n
            assert torch.equal(r, first[0]) and torch.equal(n, first[1])
        layer.forward_residual(x, logits, res, norm, gains[2], out=(res, x.clone()))
        assert torch.equal(res, first[0])


def test_a_layer_without_a_gate_takes_what_follows_too():
    from bit_mixture_experts_gb300 import ResidualNorm
    for T, impl, fuse in ((1, "auto", False), (100, "tc", True)):
        d, layer, x, logits = make(T, impl)
        layer.fuse_combine = fuse  # (the combine in the down projection's epilogue gives way)
        r, n = layer.forward_residual(x, logits, x, ResidualNorm())
        no_error()
        norm = ResidualNorm()
        want = expected(layer, T, x, norm)
        check_rows(r, want[0], want[2], STEP["bf16"], "r")
        check_rows(n, want[1], want[3], STEP["bf16"], "n")


@pytest.mark.parametrize("T,k,impl", [(1, 4, "auto"), (2, 8, "auto"), (3, 5, "gemv"), (8, 4, "auto"), (8, 8, "auto"), (8, 10, "auto"),
                                      (12, 4, "gemv"), (100, 4, "auto"), (700, 4, "tc")])
def test_a_choice_that_names_an_expert_twice(T, k, impl):
    """Rows of their own, each with the values that the expert's row has where the others differ: an expert may then
    have more rows than there are tokens."""
    import torch

    from bit_mixture_experts_gb300 import ResidualNorm
    from oracle import moe_ref
    _, layer, x, _ = make(T, impl, k=k)
    b = layer.buffers(T)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(T)).cuda()
    norm = ResidualNorm()

    def run(ids):
        ids = ids.int().cuda()
        b["y"].fill_(float("nan"))
        r, n = layer.forward_residual(x, None, x, norm, choice=(ids, w))
        no_error()
        for name, want in zip(("counts", "offsets", "perm", "inv_perm"), gate_ref.sort_assignments(ids.cpu().numpy(), 64)):
            np.testing.assert_array_equal(b[name].cpu().numpy().ravel(), want, err_msg=name)
        tiles = moe_ref.block_map(b["counts"].cpu().numpy(), b["offsets"].cpu().numpy(), T, layer.block_n_for(T))
        assert int(b["num_blocks"]) == len(tiles)
        np.testing.assert_array_equal(b["block_map"][:len(tiles)].cpu().numpy(), tiles)
        y, size = gate_ref.combined(f64(b["y"]), b["inv_perm"].cpu().numpy(), f64(w))
        want = gate_ref.residual(f64(x), y, None, None, None, norm.scale, norm.eps, norm.offset, y_size=size, terms=k + 1)
        check_rows(r, want[0], want[2], STEP["bf16"], "r")
        check_rows(n, want[1], want[3], STEP["bf16"], "n")
        return b["y"][b["inv_perm"].long()].view(T, k, -1)

    first = run((torch.arange(k) + 3).expand(T, k))
    for ids, same_as_first in ((torch.full((T, k), 3), range(k)), ((torch.arange(k) // 2 * 2 + 3).expand(T, k), range(0, k, 2)),
                               (torch.where(torch.arange(k) < 2, 3, torch.arange(k) + 20).expand(T, k), (0, 1))):
        y = run(ids)
        for j in same_as_first:
            assert torch.equal(y[:, j], first[:, ids[0, j] - 3]), j


def test_choices_out_of_range_are_reported():
    """Decode and prefill: an expert that does not exist is an error, not an access out of range."""
    import torch

    from bit_mixture_experts_gb300 import ResidualNorm, _lib
    for T in (2, 600):
        d, layer, x, logits = make(T)
        ids = torch.randint(0, 64, (T, 4), device="cuda").int()
        ids[T - 1, 3] = 64 if T == 2 else -1
        r, n = layer.forward_residual(x, None, x, ResidualNorm(), choice=(ids, torch.ones((T, 4), device="cuda")))
        torch.cuda.synchronize()
        assert _lib.moe_get_device_error() != 0
        layer.forward(x, logits)  # the next call is as ever
        no_error()


def test_refusals():
    import torch

    from bit_mixture_experts_gb300 import ExpertGate, ResidualNorm
    with pytest.raises(ValueError, match="chooses 3"):
        make(4, gate=ExpertGate(3))
    with pytest.raises(ValueError, match="bias"):
        make(4, gate=ExpertGate(4, bias=bias_of(32)))
    _, layer, x, logits = make(4, gate=ExpertGate(4))
    norm = ResidualNorm()
    for kw, what in ((dict(logits=None), "either"), (dict(logits=logits, choice=(logits, logits)), "either"),
                     (dict(logits=logits[:, :32]), "logits"), (dict(logits=logits, residual=x[:2]), "residual"),
                     (dict(logits=None, choice=(logits[:, :4].int(), logits[:, :4])), "choice")):
        with pytest.raises(ValueError, match=what):
            layer.forward_residual(x, **{"residual": x, "norm": norm, **kw})
    with pytest.raises(ValueError, match="on the device"):
        layer.forward_host(None, None, None, None)
    with pytest.raises(ValueError, match="fit"):
        layer.forward_residual(x, logits, x, norm, gate=torch.ones((3, 256), device="cuda"))


def test_a_decode_step_in_a_graph():
    import torch

    from bit_mixture_experts_gb300 import ExpertGate, ResidualNorm
    gate = ExpertGate(4, bias=bias_of(64), **KW)
    for T in (4, 300):
        _, layer, x, logits = make(T, gate=gate)
        norm = ResidualNorm(torch.rand(256, device="cuda") + 0.5)
        want = [t.clone() for t in layer.forward_residual(x, logits, x, norm)]
        g = torch.cuda.CUDAGraph()
        keep = x.clone()
        with torch.cuda.graph(g):
            out = layer.forward_residual(x, logits, x, norm)
        x.zero_()
        g.replay()
        x.copy_(keep)
        for _ in range(3):
            g.replay()
        no_error()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_a_block_with_norms_and_a_gate_served(stream):
    """Chunks, then token by token: at every step what each part gave the next against the float64 oracle."""
    import torch

    from bit_mixture_experts_gb300 import block
    shape = workloads.LayerShape(H=256, E=64, k=4, F=128)
    blk = block.synthetic(shape, q_heads=8, kv_heads=2, d=64, num_pages=24, page_size=16, device=G.torch_dev(), gated=True)
    dtype = torch.float32 if stream == "f32" else torch.bfloat16
    before, around_attention, around_experts = blk.norms
    seen = {}
    attend, forward_residual = blk.attend, blk.moe.forward_residual

    def recording_attend(x, batch, xn=None):
        seen["xn"] = xn
        seen["o"] = attend(x, batch, xn)
        return seen["o"]

    def recording_experts(xn, logits, x, norm, gate):
        seen.update(n1=xn.clone(), logits=logits, x1=x.clone())
        seen["out"] = forward_residual(xn, logits, x, norm, gate)
        return seen["out"]

    blk.attend, blk.moe.forward_residual = recording_attend, recording_experts
    gen = torch.Generator().manual_seed(3)
    prompts = [torch.randn((n, shape.H), generator=gen).to(dtype).to(G.torch_dev()) for n in (75, 9, 1)]
    steps = 0
    for x, new, kv_len, _, out in block.serve(blk, prompts, 32, 3):
        no_error()
        steps += 1
        T = len(x)
        _, want, _, dn = gate_ref.residual(f64(x), None, f64(before.w_pre))
        check_rows(seen["xn"], want, dn, STEP["bf16"], "norm before the attention")
        y = seen["o"].view(T, -1) @ blk.w_o.T
        r, n, dr, dn = gate_ref.residual(f64(x), f64(y), f64(around_attention.w_pre), f64(around_attention.w_post),
                                         f64(blk.gates[0]))
        check_rows(seen["x1"], r, dr, STEP[stream], "stream after the attention")
        check_rows(seen["n1"], n, dn, STEP["bf16"], "norm before the experts")
        g = blk.moe.gate
        ids, w = gate_ref.choose(f64(seen["logits"]).astype(np.float32), 4, score="sigmoid", bias=f64(g.bias).astype(np.float32),
                                 groups=g.groups, top_groups=g.top_groups, scale=g.scale)
        b = blk.moe.buffers(T)
        np.testing.assert_array_equal(b["topk_ids"].cpu().numpy(), ids)
        np.testing.assert_allclose(f64(b["topk_w"]), w, rtol=2e-6)
        r, n, dr, dn = expected(blk.moe, T, seen["x1"], around_experts, blk.gates[1])
        check_rows(seen["out"][0], r, dr, STEP[stream], "stream after the experts")
        check_rows(seen["out"][1], n, dn, STEP["bf16"], "norm after the experts")
        assert out.dtype == dtype and torch.equal(out, seen["out"][0]) and torch.isfinite(out).all()
    assert steps == 6
