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
from .gate import Fixed, _current_device, _empty

_F32 = {torch.bfloat16: 0, torch.float32: 1}


def _row_stride(t, name, dtype, shape, device):
    """The distance of t's rows, which must be contiguous and as the others'."""
    strides = t.stride()
    if t.shape != shape or t.dtype != dtype or t.device != device or (strides[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} on {device} with contiguous rows: got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}, strides {strides}")
    return strides[0]


class ResidualNorm(Fixed):
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
        self._constants = _lib.Residual(w_pre=_lib._ptr(w_pre), w_post=_lib._ptr(w_post), post=int(w_post is not None),
                                        param_f32=_F32[given[0].dtype] if given else 0, offset=offset, scale=scale, eps=eps)

    def describe(self, x, gate, out, stream=None, post=True):
        """The call's description for the library, and its outputs (r, n): `out`, or new ones of `stream`."""
        shape, dev, dtype = x.shape, x.device, x.dtype
        if len(shape) != 2 or not x.is_cuda or dtype not in _F32:
            raise ValueError(f"x must be bfloat16 or float32 [T, H] on a CUDA device: got {dtype} {tuple(shape)} on {dev}")
        if self.H is not None and (self.H != shape[1] or self.device != dev):
            raise ValueError(f"x is {tuple(shape)} on {dev}, the gains [{self.H}] on {self.device}")
        if _current_device() != dev.index:
            raise ValueError(f"x is on {dev}, but device {_current_device()} is the current one")
        s = _lib.Residual.from_buffer_copy(self._constants)
        s.x, s.x_stride, s.stream_f32 = x.data_ptr(), _row_stride(x, "x", dtype, shape, dev), _F32[dtype]
        if out is None:
            r, n = _empty(shape, dtype, dev, stream), _empty(shape, torch.bfloat16, dev, stream)
        else:
            r, n = out
        if r is not None:
            s.r, s.r_stride = r.data_ptr(), _row_stride(r, "out[0]", dtype, shape, dev)
        if n is not None:
            s.n, s.n_stride = n.data_ptr(), _row_stride(n, "out[1]", torch.bfloat16, shape, dev)
        if not post:
            s.post = 0
        if gate is not None:
            # [H], [1], [T, 1], [1, H] or [T, H], as broadcast against [T, H]
            dims, strides, g_type = gate.shape, gate.stride(), gate.dtype
            if len(dims) == 1:
                dims, strides = (1, dims[0]), (0, strides[0])
            if (len(dims) != 2 or g_type not in _F32 or gate.device != dev or dims[0] not in (1, shape[0])
                    or dims[1] not in (1, shape[1]) or (dims[1] > 1 and strides[1] != 1)):
                raise ValueError(f"gate must be bfloat16 or float32 on {dev}, with contiguous rows, and fit {tuple(shape)}: "
                                 f"got {g_type} {tuple(gate.shape)} on {gate.device}, strides {gate.stride()}")
            s.gate, s.gate_f32 = gate.data_ptr(), _F32[g_type]
            s.gate_per_channel = int(dims[1] > 1)
            # (one token's own row is told apart from all tokens': an output may take its place)
            s.gate_token_stride = strides[0] if dims[0] > 1 or (shape[0] == 1 and dims[1] > 1 and len(gate.shape) == 2) else 0
        return s, (r, n)

    def add(self, x, y, gate=None, out=None, stream=None):
        """(r, n) of the stream x [T, H] and the block's output y (bf16 [T, H]).  `gate`: bf16 or float32 that broadcasts
        against [T, H].  `out`: the pair to write, either of which may be None."""
        s, out = self.describe(x, gate, out, stream)
        T, H = shape = x.shape
        _lib.moe_residual_norm(y, _row_stride(y, "y", torch.bfloat16, shape, x.device), T, H, s, stream)
        return out

    def norm(self, x, out=None, stream=None):
        """n of r = scale x: the norm before a first block, bf16 [T, H] (`out` None: a new tensor)."""
        if out is None and x.is_cuda:
            out = _empty(x.shape, torch.bfloat16, x.device, stream)
        n = out
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
        _row_stride(y, "y", torch.bfloat16, (T * k + T, H), x.device)
        if not y.is_contiguous():
            raise ValueError(f"y must be contiguous: strides {y.stride()}")
        _lib.moe_combine_residual_norm(y, inv_perm, topk_w, T, H, k, s, stream)
        return out
