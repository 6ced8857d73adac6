"""The residual norms over enough rows that they go through the ring in shared memory: whole tokens or single rows as its
stages, aligned rows and others, chosen rows against the float64 oracle, and the ring's waits when they run out."""
import numpy as np
import pytest

from oracle import gate_ref
from test_residual_gpu import STEP, Case, check_rows, f64

pytestmark = pytest.mark.gpu


def setup_module():
    import gpu_util
    gpu_util.ensure_built()


def check_some(c, r, n, seed=0):
    """The first, the last and some rows in between."""
    import torch
    T, k = c.T, c.k
    rows = np.unique(np.concatenate([[0, 1, T - 2, T - 1], np.random.default_rng(seed).integers(0, T, 24)]))
    at = torch.tensor(rows, device="cuda")
    if k:
        idx = c.inv_perm.view(T, k)[at].long()
        w = f64(c.topk_w[at])
        terms = [w[:, j, None] * f64(c.y[idx[:, j]]) for j in range(k)] + [f64(c.y[T * k + at])]
        y, size = sum(terms), sum(np.abs(t) for t in terms)
    else:
        y, size = f64(c.y[at]), None
    gate = c.gate
    if gate is not None and gate.dim() == 2 and gate.shape[0] == T:
        gate = gate[at]
    want_r, want_n, dr, dn = gate_ref.residual(f64(c.x[at]), y, f64(c.w_pre), f64(c.w_post), f64(gate), c.scale, c.eps,
                                               c.offset, y_size=size, terms=k + 1)
    if r is not None:
        check_rows(r[at], want_r, dr, STEP[c.stream], "r")
    if n is not None:
        check_rows(n[at], want_n, dn, STEP["bf16"], "n")
    assert r is None or not torch.isnan(r).any()
    assert n is None or not torch.isnan(n).any()


@pytest.mark.parametrize("H", [520, 1000, 1024, 1999, 2048, 2056, 4104, 5001, 8192, 12000, 16384, 16400])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_many_rows(H, stream):
    for post, gate, gate_type in ((True, "none", "bf16"), (False, "token", "f32"), (True, "full", "bf16"),
                                  (True, "channel", "f32")):
        c = Case(3001 if H <= 2048 else 700, H, stream, post=post, gate=gate, gate_type=gate_type, scale=0.5, seed=H)
        check_some(c, *c.run())


@pytest.mark.parametrize("H,k", [(520, 1), (1001, 8), (2048, 8), (2048, 32), (4096, 8), (4096, 16), (8192, 8), (8190, 2),
                                 (16384, 3), (16384, 8)])
def test_many_combined_rows(H, k):
    for stream, gate in (("bf16", "token"), ("f32", "full")):
        c = Case(650, H, stream, gate=gate, k=k, post=k != 3, seed=k)
        check_some(c, *c.run())


@pytest.mark.parametrize("pad,shift", [(3, 0), (4, 5), (0, 1), (8, 0)])
@pytest.mark.parametrize("H", [600, 2048, 2050])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_strides_and_alignments(pad, shift, H, stream):
    import torch
    for k in (0, 2):
        c = Case(800, H, stream, pad=pad, shift=shift, gate="full", k=k)
        out = (c.rows(800, c.dtype), c.rows(800, torch.bfloat16))
        around = [o._base for o in out]
        for a in around:
            a.fill_(-3.0)
        check_some(c, *c.run(out))
        for a, o in zip(around, out):
            o.fill_(-3.0)
            assert (a == -3.0).all()  # what lies between the rows stayed as it was


@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 0), (4, 5), (8, 0)])
@pytest.mark.parametrize("H", [520, 640, 1001, 1024])
@pytest.mark.parametrize("k", [0, 2, 8])
def test_narrow_rows(H, k, pad, shift):
    """More rows than can have a block at once where blocks are small."""
    import torch
    for stream, gate in (("bf16", "full"), ("f32", "token")):
        c = Case(4900, H, stream, pad=pad, shift=shift, gate=gate, k=k, seed=H + k)
        out = (c.rows(4900, c.dtype), c.rows(4900, torch.bfloat16))
        around = [o._base for o in out]
        for a in around:
            a.fill_(-3.0)
        r, n = c.run(out)
        check_some(c, r, n)
        first = r.clone(), n.clone()
        if pad == 0 and k == 0 and stream == "bf16":
            c.run((c.y, c.x))
            assert torch.equal(c.y, first[0]) and torch.equal(c.x, first[1])
        for a, o in zip(around, out):
            o.fill_(-3.0)
            assert (a == -3.0).all()


@pytest.mark.parametrize("H", [640, 1999, 2048, 16384])
def test_outputs_left_out_and_in_place(H):
    import torch
    for post in (True, False):
        c = Case(900, H, "bf16", gate="full", post=post)
        r, n = c.run()
        a, b = torch.empty_like(r), torch.empty_like(n)
        c.run((a, None))
        c.run((None, b))
        assert torch.equal(a, r) and torch.equal(b, n)
        x, y, g = c.x.clone(), c.y.clone(), c.gate.clone()
        c.run((c.x, c.y))
        assert torch.equal(c.x, r) and torch.equal(c.y, n)
        c.x, c.y = x.clone(), y.clone()
        c.run((c.y, c.gate))
        assert torch.equal(c.y, r) and torch.equal(c.gate, n)
        c.x, c.y, c.gate = x, y.clone(), g
        assert torch.equal(c.norm.norm(x), Case.run(c, (a, b))[1]) is False  # the norm alone is something else
        only = gate_ref.residual(f64(x[:5]), None, f64(c.w_pre))
        check_rows(c.norm.norm(x)[:5], only[1], only[3], STEP["bf16"], "n")


def test_short_rows_are_the_same_however_many():
    """Rows of up to 512 channels, and the same rows in a larger call: the same bits."""
    import torch
    for H in (1, 17, 40, 64, 100, 256, 300, 512):
        for k in (0, 3):
            c = Case(5000, H, "f32", gate="token", k=0, seed=1) if k == 0 else Case(700, H, "f32", gate="token", k=k)
            r, n = c.run()
            check_some(c, r, n)
            if k == 0:
                few = c.norm.add(c.x[:7], c.y[:7], c.gate[:7])
                assert torch.equal(few[0], r[:7]) and torch.equal(few[1], n[:7])


@pytest.mark.parametrize("H", [2048, 12000])
def test_rows_that_are_not_finite_stay_alone(H):
    import torch
    c = Case(1300, H, "bf16", k=2)
    r, n = c.run()
    c.x[7, 3] = float("nan")
    c.y[c.inv_perm[2 * 900].long(), 5] = float("inf")
    a, b = c.run()
    keep = torch.ones(1300, dtype=torch.bool, device="cuda")
    keep[[7, 900]] = False
    assert torch.equal(a[keep], r[keep]) and torch.equal(b[keep], n[keep])
    assert torch.isnan(b[7]).all() and torch.isnan(b[900, 5])


@pytest.mark.parametrize("H,k", [(2048, 2), (16384, 8)])
def test_bad_rows_are_skipped_and_reported(H, k):
    import torch

    from bit_mixture_experts_gb300 import _lib
    c = Case(640, H, "bf16", k=k, post=False)
    bad = c.inv_perm.clone()
    bad[[3 * k, 3 * k + 1, 639 * k]] = torch.tensor([-5, 640 * k, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    zero = c.topk_w.clone()
    zero.view(-1)[[3 * k, 3 * k + 1, 639 * k]] = 0
    idx, w = c.inv_perm, c.topk_w
    c.topk_w = zero
    want = c.run()
    c.inv_perm, c.topk_w = bad, w
    got = c.run()
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 2
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_graphs_of_one_norm():
    import torch
    c = Case(1000, 2048, "bf16", k=4)
    r, n = c.run()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.run())
        graphs.append(g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs[0].replay()
    with torch.cuda.stream(side):
        graphs[1].replay()
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, r) and torch.equal(b, n)


def test_waits_that_run_out_are_reported():
    """A limit of a nanosecond, and many more rows per block than stages (so that the copying warp has to wait for one):
    the call ends, and says so; the next one is as ever."""
    import torch

    from bit_mixture_experts_gb300 import _lib
    for H, k in ((2048, 4), (1999, 0), (16384, 8)):
        c = Case(20000 if H < 4096 else 700, H, "bf16", k=k)
        r, n = c.run()
        torch.cuda.synchronize()
        assert _lib.moe_get_device_error() == 0
        _lib.moe_set_wait_limit_ns(1)
        try:
            c.run()
            torch.cuda.synchronize()
            assert _lib.moe_get_device_error() == 3
        finally:
            _lib.moe_set_wait_limit_ns(1_000_000_000)
        a, b = c.run()
        torch.cuda.synchronize()
        assert _lib.moe_get_device_error() == 0
        assert torch.equal(a, r) and torch.equal(b, n)
