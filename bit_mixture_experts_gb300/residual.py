"""The norms around a block's residual addition, in one launch:

    z = y / rms(y) * (w_post + offset)     (y itself without w_post)
    r = scale x + gate z                   the residual stream's next value
    n = r / rms(r) * (w_pre + offset)      what the next block takes

``add`` takes the block's output y as it is, ``combine`` as the rows of a token's experts, ``norm`` is for where no block
has come before.  PyTorch only provides device memory and the stream.
"""
from __future__ import annotations

import torch

from . import _lib
from .gate import _on

_F32 = {torch.bfloat16: 0, torch.float32: 1}


class ResidualNorm:
    """w_pre, w_post: bf16 or float32 [H] (both of one type); w_post None: the block's output is not normed, w_pre None:
    gains of 1.  The stream x is bf16 or float32, r has its type; y and n are bf16.  Tensors are [T, H] with rows of any
    stride; r may be x's or y's memory and n x's or y's, where type and strides are the same."""

    def __init__(self, w_pre=None, w_post=None, scale=1.0, eps=1e-6, offset=0.0):
        _lib.load()
        given = [w for w in (w_pre, w_post) if w is not None]
        for w in given:
            if w.dtype not in _F32 or w.dtype != given[0].dtype or w.dim() != 1 or not w.is_contiguous() \
                    or w.device.type != "cuda" or w.shape != given[0].shape or w.device != given[0].device:
                raise ValueError("w_pre and w_post must be contiguous bfloat16 or float32 vectors, alike, on a CUDA "
                                 f"device: got {[(w.dtype, tuple(w.shape), str(w.device)) for w in given]}")
        self.w_pre, self.w_post, self.scale, self.eps, self.offset = w_pre, w_post, scale, eps, offset
        self.H = given[0].shape[0] if given else None
        self.device = given[0].device if given else None
        self.param_f32 = _F32[given[0].dtype] if given else 0

    def _rows(self, t, name, dtypes, shape, device):
        if t.dtype not in dtypes or t.shape != shape or t.device != device or (t.stride(1) != 1 and shape[1] > 1):
            raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)} {tuple(shape)} on {device} with "
                             f"contiguous rows: got {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}")

    def describe(self, x, gate, out, stream=None, post=True):
        """The call's description for the library, and its outputs (r, n): `out`, or new ones of `stream`."""
        if x.dim() != 2 or x.device.type != "cuda":
            raise ValueError(f"x must be [T, H] on a CUDA device: got {tuple(x.shape)} on {x.device}")
        shape, dev = x.shape, x.device
        self._rows(x, "x", tuple(_F32), shape, dev)
        if self.H is not None and (self.H != shape[1] or self.device != dev):
            raise ValueError(f"x is {tuple(shape)} on {dev}, the gains [{self.H}] on {self.device}")
        if torch.cuda.current_device() != dev.index:
            raise ValueError(f"x is on {dev}, but device {torch.cuda.current_device()} is the current one")
        if out is None:
            with _on(stream, dev):
                r, n = torch.empty(shape, dtype=x.dtype, device=dev), torch.empty(shape, dtype=torch.bfloat16, device=dev)
        else:
            r, n = out
            if r is not None:
                self._rows(r, "out[0]", (x.dtype,), shape, dev)
            if n is not None:
                self._rows(n, "out[1]", (torch.bfloat16,), shape, dev)
        g_ptr, g_token, g_channel, g_f32 = None, 0, 0, 0
        if gate is not None:
            # [H], [1], [T, 1], [1, H] or [T, H], as broadcast against [T, H]
            g = gate if gate.dim() == 2 else gate[None]
            if (gate.dim() not in (1, 2) or g.dtype not in _F32 or g.device != dev
                    or g.shape[0] not in (1, shape[0]) or g.shape[1] not in (1, shape[1])
                    or (g.shape[1] > 1 and g.stride(1) != 1)):
                raise ValueError(f"gate must be bfloat16 or float32 on {dev}, with contiguous rows, and fit {tuple(shape)}: "
                                 f"got {gate.dtype} {tuple(gate.shape)} on {gate.device}, strides {gate.stride()}")
            g_ptr, g_f32 = g.data_ptr(), _F32[g.dtype]
            g_token, g_channel = g.stride(0) if g.shape[0] > 1 else 0, int(g.shape[1] > 1)
        s = _lib.Residual(x.data_ptr(), x.stride(0), _lib._ptr(r), 0 if r is None else r.stride(0), _lib._ptr(n),
                          0 if n is None else n.stride(0), _lib._ptr(self.w_pre), _lib._ptr(self.w_post), g_ptr, g_token,
                          g_channel, int(post and self.w_post is not None), _F32[x.dtype], self.param_f32, g_f32,
                          self.offset, self.scale, self.eps)
        return s, (r, n)

    def add(self, x, y, gate=None, out=None, stream=None):
        """(r, n) of the stream x [T, H] and the block's output y (bf16 [T, H]).  `gate`: bf16 or float32 that broadcasts
        against [T, H].  `out`: the pair to write, either of which may be None."""
        s, out = self.describe(x, gate, out, stream)
        self._rows(y, "y", (torch.bfloat16,), x.shape, x.device)
        _lib.moe_residual_norm(y, y.stride(0), x.shape[0], x.shape[1], s, stream)
        return out

    def norm(self, x, out=None, stream=None):
        """n of r = scale x: the norm before a first block, bf16 [T, H] (`out` None: a new tensor)."""
        with _on(stream, x.device):
            n = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device) if out is None else out
        s, _ = self.describe(x, None, (None, n), stream, post=False)
        _lib.moe_residual_norm(None, 0, x.shape[0], x.shape[1], s, stream)
        return n

    def combine(self, x, y, inv_perm, topk_w, gate=None, out=None, stream=None):
        """``add`` where a token's y is the weighted sum of its experts' rows and its shared expert's: y bf16
        [T k + T, H], inv_perm int32 [T k], topk_w float32 [T, k], as the routing and the down projection give them."""
        s, out = self.describe(x, gate, out, stream)
        T, H = x.shape
        k = topk_w.shape[-1]
        if topk_w.dtype != torch.float32 or topk_w.shape != (T, k) or topk_w.device != x.device or not topk_w.is_contiguous():
            raise ValueError(f"topk_w must be contiguous float32 [{T}, k] on {x.device}: got {topk_w.dtype} "
                             f"{tuple(topk_w.shape)} on {topk_w.device}")
        if inv_perm.dtype != torch.int32 or inv_perm.numel() != T * k or inv_perm.device != x.device \
                or not inv_perm.is_contiguous():
            raise ValueError(f"inv_perm must be contiguous int32 [{T * k}] on {x.device}: got {inv_perm.dtype} "
                             f"{tuple(inv_perm.shape)} on {inv_perm.device}")
        self._rows(y, "y", (torch.bfloat16,), (T * k + T, H), x.device)
        if not y.is_contiguous():
            raise ValueError(f"y must be contiguous: strides {y.stride()}")
        _lib.moe_combine_residual_norm(y, inv_perm, topk_w, T, H, k, s, stream)
        return out
