"""moe_residual_norm and moe_combine_residual_norm on the GPU against the float64 oracle: every element of r and n within
the bound of its FP32 arithmetic and one rounding."""
import numpy as np
import pytest

from oracle import gate_ref

pytestmark = pytest.mark.gpu

STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # a rounding, relative


def setup_module():
    import gpu_util
    gpu_util.ensure_built()


def types():
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


class Case:
    """Inputs of one call; `pad`: elements between rows, `shift`: of the first row from an aligned address."""

    def __init__(self, T, H, stream="bf16", param="bf16", gate="none", gate_type="bf16", post=True, pre=True, scale=1.0,
                 offset=0.0, pad=0, shift=0, k=0, seed=0, eps=1e-6):
        import torch

        from bit_mixture_experts_gb300 import ResidualNorm
        gen = torch.Generator(device="cuda").manual_seed(seed + T * 31 + H)
        dt = types()

        def normal(*shape):
            return torch.randn(shape, generator=gen, device="cuda")

        def rows(n, dtype, loose=True):
            p, s = (pad, shift) if loose else (0, 0)
            x = torch.full((n * (H + p) + s,), float("nan"), dtype=dtype, device="cuda")[s:].view(n, H + p)[:, :H]
            x.copy_(normal(n, H) * torch.exp(normal(n, 1)))
            return x

        self.T, self.H, self.k, self.eps, self.scale, self.offset = T, H, k, eps, scale, offset
        self.stream, self.dtype = stream, dt[stream]
        self.x = rows(T, dt[stream])
        self.y = rows(T * (k + 1), torch.bfloat16, loose=k == 0)
        self.w_pre = (normal(H) * 0.3 + 1).to(dt[param]) if pre else None
        self.w_post = (normal(H) * 0.3 + 1).to(dt[param]) if post else None
        shape = {"none": None, "one": (1,), "channel": (H,), "row": (1, H), "token": (T, 1), "full": (T, H)}[gate]
        self.gate = None if shape is None else (normal(*shape) * 0.5).to(dt[gate_type])
        if k:
            self.inv_perm = torch.randperm(T * k, generator=gen, device="cuda").int()
            self.topk_w = normal(T, k)
        self.norm = ResidualNorm(self.w_pre, self.w_post, scale, eps, offset)
        self.rows = rows

    def run(self, out=None, stream=None):
        if self.k:
            return self.norm.combine(self.x, self.y, self.inv_perm, self.topk_w, self.gate, out, stream)
        return self.norm.add(self.x, self.y, self.gate, out, stream)

    def want(self):
        y, size = f64(self.y), None
        if self.k:
            y, size = gate_ref.combined(y, self.inv_perm.cpu().numpy(), f64(self.topk_w))
        return gate_ref.residual(f64(self.x), y, f64(self.w_pre), f64(self.w_post), f64(self.gate), self.scale, self.eps,
                                 self.offset, y_size=size, terms=self.k + 1)


def check_rows(got, ref, bound, step, what):
    off = np.abs(f64(got) - ref) - (bound + step * (np.abs(ref) + bound))
    assert not np.isnan(off).any(), what
    assert (off <= 0).all(), (what, float(off.max()))


def check(c, r, n, want=None):
    ref_r, ref_n, dr, dn = want or c.want()
    if r is not None:
        check_rows(r, ref_r, dr, STEP[c.stream], "r")
    if n is not None:
        check_rows(n, ref_n, dn, STEP["bf16"], "n")


SIZES = [(1, 1), (1, 8), (3, 7), (2, 64), (9, 256), (5, 257), (17, 512), (4, 520), (33, 1024), (3, 1999), (1, 2048),
         (7, 4104), (2, 8192), (3, 8200), (2, 16384), (2, 16392), (1, 32768), (2, 32767)]


@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", SIZES)
def test_sizes(T, H, stream):
    for k in (0, 3):
        for post in (True, False):
            c = Case(T, H, stream, post=post, k=k, gate="channel" if post else "none")
            check(c, *c.run())


@pytest.mark.parametrize("gate", ["none", "one", "channel", "row", "token", "full"])
@pytest.mark.parametrize("gate_type,param", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("H", [200, 1000, 2048, 777])
def test_gates_and_types(gate, gate_type, param, H):
    for stream, k in (("bf16", 0), ("f32", 0), ("bf16", 8)):
        c = Case(6, H, stream, param, gate, gate_type, k=k, scale=0.7071, offset=1.0 if param == "f32" else 0.0, seed=3)
        check(c, *c.run())


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (4, 0), (3, 0), (1, 1), (0, 3), (64, 4)])
@pytest.mark.parametrize("H", [64, 250, 1024, 2056])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_strides_and_alignments(pad, shift, H, stream):
    import torch
    c = Case(5, H, stream, pad=pad, shift=shift, gate="token")
    out = (c.rows(5, c.dtype), c.rows(5, torch.bfloat16))
    # what lies between the rows stays as it was
    around = [o._base if o._base is not None else o for o in out]
    for a in around:
        a.fill_(-3.0)
    got = c.run(out)
    assert got[0] is out[0]
    check(c, *got)
    for a, o in zip(around, out):
        o.fill_(-3.0)
        assert (a == -3.0).all()


def test_outputs_left_out():
    for stream in ("bf16", "f32"):
        c = Case(7, 512, stream)
        r, n = c.run()
        import torch
        a, b = torch.empty_like(r), torch.empty_like(n)
        c.run((a, None))
        c.run((None, b))
        assert torch.equal(a, r) and torch.equal(b, n)


@pytest.mark.parametrize("H", [256, 300, 2048, 20000])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_in_place(H, stream):
    import torch
    c = Case(9, H, stream, gate="full", gate_type="bf16")
    r, n = c.run()
    x, y, g = c.x.clone(), c.y.clone(), c.gate.clone()
    c.run((c.x, c.y))  # r in x's place, n in y's
    assert torch.equal(c.x, r) and torch.equal(c.y, n)
    c.x, c.y = x.clone(), y.clone()
    c.run((c.x, c.gate))  # n in the gate's place
    assert torch.equal(c.x, r) and torch.equal(c.gate, n)
    if stream == "bf16":
        c.x, c.y, c.gate = x.clone(), y.clone(), g.clone()
        c.run((c.y, c.x))  # crossed over
        assert torch.equal(c.y, r) and torch.equal(c.x, n)
    # columns of one wider tensor
    wide = torch.empty((9, 2 * H), dtype=torch.bfloat16, device="cuda")
    if stream == "bf16":
        wide[:, :H] = x
        c.x, c.y, c.gate = wide[:, :H], y, g
        c.run((wide[:, :H], wide[:, H:]))
        assert torch.equal(wide[:, :H], r) and torch.equal(wide[:, H:], n)


def test_one_row_for_all_tokens():
    c = Case(6, 640, "f32")
    c.x, c.y = c.x[:1].expand(6, -1), c.y[:1].expand(6, -1)
    check(c, *c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_alone(dtype):
    import torch

    from bit_mixture_experts_gb300 import ResidualNorm, _lib
    for T, H in ((1, 2048), (5, 333), (0, 64)):
        x = torch.randn((T, H), device="cuda").to(types()[dtype])
        w = torch.randn(H, device="cuda")
        n = ResidualNorm(w, w, scale=0.5, offset=1.0).norm(x)  # w_post has no part in it
        if T:
            _, ref, _, dn = gate_ref.residual(f64(x), None, f64(w), scale=0.5, offset=1.0)
            check_rows(n, ref, dn, STEP["bf16"], "n")
    # without gains it is moe_rms_norm
    x = torch.randn((33, 2048), device="cuda").bfloat16()
    old = torch.empty_like(x)
    _lib.moe_rms_norm(x, old)
    _, ref, _, dn = gate_ref.residual(f64(x), None)
    for n in (ResidualNorm().norm(x), old):
        check_rows(n, ref, dn, STEP["bf16"], "n")


@pytest.mark.parametrize("H", [320, 2048, 1001])
def test_rows_that_are_zero_or_not_finite(H):
    import torch
    for k in (0, 2):
        c = Case(6, H, "f32", k=k, gate="none")
        rows = [c.inv_perm[k:2 * k].long().tolist() + [6 * k + 1] if k else [1]][0]
        want_clean = c.want()
        c.x[1] = 0
        c.y[rows] = 0  # a token whose stream is zero: zeros, not NaN
        c.x[2, 5] = float("inf")
        c.x[3, H - 1] = float("nan")
        r, n = c.run()
        assert (r[1] == 0).all() and (n[1] == 0).all()
        assert r[2, 5] == float("inf") and torch.isnan(n[2, 5])
        assert torch.isnan(r[3, H - 1]) and torch.isnan(n[3]).all()
        rest = [0, 4, 5]  # other tokens take no notice
        check(c, r[rest], n[rest], [a[rest] for a in want_clean])


def test_bad_rows_are_skipped_and_reported():
    import torch

    from bit_mixture_experts_gb300 import _lib
    c = Case(4, 256, "bf16", k=2, post=False)
    c.inv_perm[1], c.inv_perm[6] = -1, 1 << 30
    r, n = c.run()
    torch.cuda.synchronize()
    assert _lib.moe_get_device_error() == 2
    y, w = f64(c.y), f64(c.topk_w)
    w.reshape(-1)[[1, 6]] = 0
    idx = c.inv_perm.cpu().numpy().copy()
    idx[[1, 6]] = 0
    y, size = gate_ref.combined(y, idx, w)
    check(c, r, n, gate_ref.residual(f64(c.x), y, f64(c.w_pre), y_size=size, terms=3))


def test_streams_and_graphs():
    import torch
    for k in (0, 4):
        c = Case(300, 2048, "bf16", k=k, gate="channel")
        r, n = c.run()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for s in (side, side.cuda_stream):
            a, b = c.run(stream=s)
            side.synchronize()
            assert torch.equal(a, r) and torch.equal(b, n)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = c.run()
        x = c.x.clone()
        c.x.zero_()
        g.replay()
        c.x.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], r) and torch.equal(out[1], n)


def test_combine_is_the_norm_of_the_sum():
    """With weights and rows whose sums are exact in bf16, the fused call gives the bits of moe_combine and add."""
    import torch

    from bit_mixture_experts_gb300 import _lib
    c = Case(50, 512, "f32", k=4, gate="token")
    c.y.copy_(torch.randint(-8, 9, c.y.shape, device="cuda"))
    c.topk_w.copy_(torch.randint(-2, 3, c.topk_w.shape, device="cuda"))
    r, n = c.run()
    y = torch.empty((50, 512), dtype=torch.bfloat16, device="cuda")
    _lib.moe_combine(c.y, c.inv_perm, c.topk_w, y)
    a, b = c.norm.add(c.x, y, c.gate)
    assert torch.equal(a, r) and torch.equal(b, n)
