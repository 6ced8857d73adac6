"""A paged key/value cache and the attention that reads it, driven through the C ABI.

One pool of pages serves many sequences.  A step's batch is described once (``PagedKVCache.batch``) and
shared by the three calls of the step: ``append`` writes the new tokens' keys and values (bf16, or quantised
to e4m3 with one power-of-two scale per token and head), ``attention`` attends from the new tokens to
everything their sequence has cached, ``read`` returns what the cache holds for them.  PyTorch only provides
device memory and the stream; every step runs in libmoe_w4.so's kernels.
"""
from __future__ import annotations

import torch

from . import _lib

FORMATS = {"bf16": _lib.KV_BF16, "e4m3": _lib.KV_E4M3}


class KVBatch:
    """One step's sequences (see ``PagedKVCache.batch``).  Holds the index tensors, whose contents may change
    between calls; the sizes may not."""

    def __init__(self, page_table, cu_q, kv_len, T, device):
        for name, t, nd in (("page_table", page_table, 2), ("cu_q", cu_q, 1), ("kv_len", kv_len, 1)):
            if t.dtype != torch.int32 or t.dim() != nd or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 tensor of {nd} dimension(s)")
            if t.device != device:
                raise ValueError(f"{name} is on {t.device}, the cache on {device}")
        B, width = page_table.shape
        if cu_q.shape[0] != B + 1 or kv_len.shape[0] != B:
            raise ValueError(f"{B} sequences in page_table need cu_q of {B + 1} and kv_len of {B} elements")
        self.T = int(T)
        self.workspace = {}  # bytes of scratch that an attention needs, by cache and query heads
        self.tensors = (page_table, cu_q, kv_len)
        self.struct = _lib.KVBatch(page_table.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(), B, width, self.T)


class PagedKVCache:
    """Pages of `page_size` tokens of `heads` KV heads of `d` values, for keys and for values.

    ``fmt`` "bf16" keeps the values as they are; "e4m3" keeps 8-bit floats and a float32 scale (a power of
    two) per token and head.  ``k`` and ``v`` have shape [num_pages, heads, page_size, d], ``k_scale`` and
    ``v_scale`` [num_pages, heads, page_size].
    """

    def __init__(self, num_pages, page_size, heads, d, fmt="bf16", device="cuda"):
        if fmt not in FORMATS:
            raise ValueError(f"fmt {fmt!r} is none of {sorted(FORMATS)}")
        shape = (num_pages, heads, page_size, d)
        dtype = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        scales = (None, None)
        if fmt == "e4m3":
            scales = tuple(torch.empty(shape[:3], dtype=torch.float32, device=device) for _ in range(2))
        self._init(k, v, *scales)

    @classmethod
    def from_tensors(cls, k, v, k_scale=None, v_scale=None):
        """A cache over existing pools (e4m3 when they are float8_e4m3fn; scales must be powers of two)."""
        self = cls.__new__(cls)
        self._init(k, v, k_scale, v_scale)
        return self

    def _init(self, k, v, k_scale, v_scale):
        _lib.load()
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError(f"pages must be bfloat16 or float8_e4m3fn, not {k.dtype}")
        if k.device.type != "cuda":
            raise ValueError(f"the cache's tensors must be on a CUDA device, not on {k.device}")
        self.fmt = "bf16" if k.dtype == torch.bfloat16 else "e4m3"
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype or v.device != k.device:
            raise ValueError("k and v must be alike: [num_pages, heads, page_size, d]")
        pools = [k, v]
        if self.fmt == "e4m3":
            for s in (k_scale, v_scale):
                if s is None or s.dtype != torch.float32 or s.shape != k.shape[:3] or s.device != k.device:
                    raise ValueError("an e4m3 cache needs float32 k_scale and v_scale [num_pages, heads, page_size]")
            pools += [k_scale, v_scale]
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
        if not all(t.is_contiguous() for t in pools):
            raise ValueError("the cache's tensors must be contiguous")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.device_index = k.device, k.device.index
        self.num_pages, self.heads, self.page_size, self.d = k.shape
        self._workspaces = {}
        self.struct = _lib.KVCache(k.data_ptr(), v.data_ptr(), _lib._ptr(k_scale), _lib._ptr(v_scale), self.num_pages,
                                   self.page_size, self.heads, self.d, FORMATS[self.fmt])

    def batch(self, page_table, cu_q, kv_len, T):
        """Sequence b's new tokens are rows cu_q[b] .. cu_q[b+1]-1 of a step's T rows; kv_len[b] counts its
        tokens with the new ones; position p lives in page page_table[b, p // page_size].  All int32 on the
        cache's device; they are read by the kernels, never by the host."""
        return KVBatch(page_table, cu_q, kv_len, T, self.device)

    def _rows(self, t, name, batch, heads=None):
        """Checks a [T, heads, d] bf16 tensor whose rows of d are contiguous."""
        sh = t.shape
        if (t.dtype != torch.bfloat16 or len(sh) != 3 or sh[0] != batch.T or sh[2] != self.d
                or (heads is not None and sh[1] != heads) or t.device != self.device
                or (t.stride(2) != 1 and t.numel() > 0)):
            want = "heads" if heads is None else heads
            raise ValueError(f"{name} must be bfloat16 [{batch.T}, {want}, {self.d}] on {self.device} with contiguous "
                             f"rows: got {t.dtype} {tuple(sh)} on {t.device}, strides {t.stride()}")

    def _check_device(self):
        """Kernels are launched on the current device: it must be the cache's."""
        if torch.cuda.current_device() != self.device_index:
            raise ValueError(f"the cache is on {self.device}, but device {torch.cuda.current_device()} is the current one")

    def _on(self, stream):
        """Makes `stream`, a torch stream or a raw handle, the current one for a `with` block."""
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.device)
        return torch.cuda.stream(stream)

    def _empty(self, shape, dtype, stream):
        """An output for a call on `stream`: allocated as memory of that stream."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with self._on(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _workspace(self, batch, q_heads, stream):
        """The attention's scratch for a call on `stream`, a tensor or (pointer, bytes).  Calls outside graph
        captures have one per stream, which grows to the largest call's need.  A call that torch.cuda.graph
        captures has its own, from the graph's memory: no later call frees or shares what the graph's replays
        write to."""
        need = batch.workspace.get((self, q_heads))
        if need is None:
            need = max(_lib.moe_kv_attention_workspace_size(self.struct, batch.struct, q_heads), 16)
            batch.workspace[(self, q_heads)] = need
        if self._capturing(stream):
            return self._empty((need,), torch.uint8, stream)
        key = _lib._stream(stream)
        have = self._workspaces.get(key)
        if have is None or have[1][1] < need:
            t = self._empty((need,), torch.uint8, stream)
            have = self._workspaces[key] = (t, (t.data_ptr(), t.nbytes))
        return have[1]

    def _capturing(self, stream):
        """Whether calls on `stream` are being captured into a graph."""
        if stream is None:
            return torch.cuda.is_current_stream_capturing()
        with self._on(stream):
            return torch.cuda.is_current_stream_capturing()

    def append(self, k, v, batch, stream=None):
        """Write the new tokens' keys and values (bf16 [T, heads, d], strided views welcome) into the cache."""
        self._check_device()
        self._rows(k, "k", batch, self.heads)
        self._rows(v, "v", batch, self.heads)
        _lib.moe_kv_append(k, v, self.struct, batch.struct, stream)

    def read(self, batch, out=None, stream=None):
        """What the cache holds at the new tokens' positions: bf16 (k, v), each [T, heads, d]."""
        self._check_device()
        if out is None:
            shape = (batch.T, self.heads, self.d)
            out = (self._empty(shape, torch.bfloat16, stream), self._empty(shape, torch.bfloat16, stream))
        else:
            for t, name in zip(out, ("out[0]", "out[1]")):
                self._rows(t, name, batch, self.heads)
                if not t.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
        _lib.moe_kv_read(out[0], out[1], self.struct, batch.struct, stream)
        return out

    def attention(self, q, batch, scale=None, out=None, return_lse=False, stream=None, workspace=None):
        """Causal attention of the new tokens' queries (bf16 [T, q_heads, d]) over their sequences' caches.

        q_heads is a multiple of the cache's heads; scale defaults to 1/sqrt(d).  Returns bf16
        [T, q_heads, d], with ``return_lse`` also the scores' natural log-sum-exp, float32 [T, q_heads]
        (-inf for a token that sees no key; its output is 0).  `workspace` (uint8, at least
        ``moe_kv_attention_workspace_size``) replaces the cache's own scratch of the stream.

        In a ``torch.cuda.graph`` capture scratch and outputs come from the graph's memory.  A capture made in
        another way has no memory of its own: give it `workspace` and `out`, keep them as long as the graph,
        and replay no two graphs that were given the same ones at the same time."""
        self._check_device()
        self._rows(q, "q", batch)
        if out is None:
            out = (torch.empty_like(q, memory_format=torch.contiguous_format) if stream is None
                   else self._empty(q.shape, torch.bfloat16, stream))
        else:
            self._rows(out, "out", batch, q.shape[1])
            if not out.is_contiguous():
                raise ValueError("out must be contiguous")
        lse = self._empty(q.shape[:2], torch.float32, stream) if return_lse else None
        if workspace is None:
            workspace = self._workspace(batch, q.shape[1], stream)
        elif torch.is_tensor(workspace) and (workspace.device != self.device or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be contiguous on {self.device}: it is on {workspace.device}, strides "
                             f"{workspace.stride()}")
        _lib.moe_kv_attention(q, self.d ** -0.5 if scale is None else scale, self.struct, batch.struct, out, lse,
                              workspace, stream)
        return (out, lse) if return_lse else out
