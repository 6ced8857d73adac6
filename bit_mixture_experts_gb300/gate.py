"""Gates: from router logits to each token's experts and their weights, in the ways that models differ.

``MoELayerW4`` and ``DecoderBlockW4`` take an ``ExpertGate``; without one they choose by the softmax that is
renormalised over the chosen.  PyTorch only provides device memory and the stream.
"""
from __future__ import annotations

import collections

import torch

from . import _lib

Routing = collections.namedtuple("Routing", "topk_ids topk_w counts offsets perm inv_perm block_map num_blocks")


def _current_device():
    """torch.cuda.current_device(), whose check that CUDA is initialised the tensors at hand make needless."""
    return torch._C._cuda_getDevice()


def _on(stream, device):
    """A `with` block in which `stream`, a torch stream or a raw handle, is the current one."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream):
    """An output for a call on `stream` (None: the current one): memory of that stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def _in_a_graphs_pool(t):
    """Whether t, made during a capture, is memory that PyTorch keeps for the graph: so in its own captures alone."""
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return tuple(s.get("segment_pool_id", (0, 0))) != (0, 0)
    return False


class Fixed:
    """An object whose description the library has been given: its public attributes keep their values.  (The memory
    of a tensor put in another's place would not be what the calls read.)"""

    def __setattr__(self, name, value):
        if name[0] != "_" and name in self.__dict__:
            raise AttributeError(f"{type(self).__name__}.{name} is fixed: make another {type(self).__name__}, or change a "
                                 "tensor's values in place")
        super().__setattr__(name, value)


class ExpertGate(Fixed):
    """Chooses k experts of a token by score plus bias, of the groups that stay, and weighs them by score.

    score    "softmax" (over all experts) or "sigmoid" of the logits
    bias     float32 [E] on the device, added to the scores for the choice alone, or None.  It is read by every
             call: a program that balances its experts' load may change it in place
    groups, top_groups, group_score
             the experts in order form `groups` groups, of which the top_groups best stay (default: all); a
             group's score is its experts' largest score plus bias ("max") or the sum of the two largest ("top2")
    renorm   weights divided by their sum;  scale: what they are multiplied by then

    Equal ones go to the lower index.  An expert whose logit is -inf or NaN is not available: it is chosen only
    where fewer than k are, with weight 0.
    """

    def __init__(self, k, score="softmax", bias=None, groups=1, top_groups=None, group_score="top2", renorm=True,
                 scale=1.0):
        _lib.load()
        if score not in _lib.SCORES:
            raise ValueError(f"score {score!r} is none of {sorted(_lib.SCORES)}")
        if group_score not in _lib.GROUP_SCORES:
            raise ValueError(f"group_score {group_score!r} is none of {sorted(_lib.GROUP_SCORES)}")
        if bias is not None and (bias.dtype != torch.float32 or bias.dim() != 1 or not bias.is_contiguous()
                                 or bias.device.type != "cuda"):
            raise ValueError(f"bias must be a contiguous float32 vector on a CUDA device: got {bias.dtype} "
                             f"{tuple(bias.shape)} on {bias.device}")
        self.k, self.score, self.bias, self.groups = k, score, bias, groups
        self.top_groups = groups if top_groups is None else top_groups
        self.group_score, self.renorm, self.scale = group_score, renorm, scale
        self._workspaces, self._plans = {}, {}
        self._captured = []  # scratch of captures that PyTorch did not begin, and keeps none for
        self.struct = _lib.Gate(_lib._ptr(bias), _lib.SCORES[score], groups, self.top_groups,
                                _lib.GROUP_SCORES[group_score], int(renorm), scale)

    def check(self, E, device):
        """Raises ValueError unless the gate fits E experts on `device`."""
        if self.bias is not None and (self.bias.shape[0] != E or self.bias.device != device):
            raise ValueError(f"the gate's bias is [{self.bias.shape[0]}] on {self.bias.device}, the logits have {E} "
                             f"experts on {device}")

    def _logits(self, logits):
        if logits.dtype != torch.float32 or logits.dim() != 2 or not logits.is_contiguous() or not logits.is_cuda:
            raise ValueError(f"logits must be contiguous float32 [T, E] on a CUDA device: got {logits.dtype} "
                             f"{tuple(logits.shape)}, strides {logits.stride()}, on {logits.device}")
        self.check(logits.shape[1], logits.device)
        if _current_device() != logits.get_device():
            raise ValueError(f"the logits are on {logits.device}, but device {_current_device()} is the current one")

    def choose(self, logits, out=None, stream=None):
        """logits float32 [T, E] -> (int32 [T, k], float32 [T, k]), or into `out`, a pair of such tensors."""
        self._logits(logits)
        shape, dev = (logits.shape[0], self.k), logits.device
        if out is None:
            out = _empty(shape, torch.int32, dev, stream), _empty(shape, torch.float32, dev, stream)
        else:
            ids, w = out
            for t, dtype in (ids, torch.int32), (w, torch.float32):
                if t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
                    raise ValueError(f"out must be contiguous int32 and float32 {shape} on {dev}: got {t.dtype} "
                                     f"{tuple(t.shape)} on {t.device}, strides {t.stride()}")
        _lib.moe_gate(logits, self.k, self.struct, out[0], out[1], stream)
        return out

    def route(self, logits, block_n, stream=None):
        """The choice and what the grouped expert GEMMs need of it: a ``Routing`` of moe_route's outputs for tiles of
        block_n rows (include/moe_w4.h).  Scratch is kept per stream, in a graph capture it is the graph's."""
        self._logits(logits)
        (T, E), k, dev = logits.shape, self.k, logits.device
        shapes, need = self._plan(T, E, block_n)
        r = Routing(*(_empty(shape, dtype, dev, stream) for shape, dtype in shapes))
        ws = self._workspace(need, stream, dev) if need else None
        _lib.moe_route_gated(logits, T, E, k, self.struct, block_n, *r, ws, stream)
        return r

    def _plan(self, T, E, block_n):
        """Shapes and types of a Routing's tensors, bytes of scratch."""
        have = self._plans.get((T, E, block_n))
        if have is None:
            A, cap, i32 = T * self.k, _lib.moe_block_map_capacity(T, E, self.k, block_n), torch.int32
            shapes = (((T, self.k), i32), ((T, self.k), torch.float32), ((E,), i32), ((E + 1,), i32), ((A,), i32),
                      ((A,), i32), ((cap, 3), i32), ((1,), i32))
            have = self._plans[T, E, block_n] = shapes, _lib.moe_route_workspace_size(T, E, self.k, block_n)
        return have

    def _workspace(self, need, stream, dev):
        """Zeros, which every call leaves behind as it found them."""
        if stream is not None:
            with _on(stream, dev):
                return self._workspace_here(need, dev)
        return self._workspace_here(need, dev)

    def _workspace_here(self, need, dev):
        if torch.cuda.is_current_stream_capturing():
            own = torch.zeros(need, dtype=torch.uint8, device=dev)
            if not _in_a_graphs_pool(own):
                self._captured.append(own)
            return own
        key = (dev, _lib._stream())
        have = self._workspaces.get(key)
        if have is None or have.numel() < need:
            have = self._workspaces[key] = torch.zeros(need, dtype=torch.uint8, device=dev)
        return have
