"""GB300-native (sm_103a) forward of a mixture-of-experts FFN layer with
groupwise-affine 4-bit expert weights and GPU-resident routing.

The kernels live in libmoe_w4.so (csrc/, C ABI in include/moe_w4.h); this
package only binds them (``_lib``) and wraps one layer (``layer.MoELayerW4``),
the gates that choose a layer's experts (``gate.ExpertGate``), the norms around
a block's residual addition (``residual.ResidualNorm``) and the paged key/value
cache with its attention (``kv.PagedKVCache``).
"""
from . import _lib  # noqa: F401
from ._lib import MoeError, load  # noqa: F401

__all__ = ["MoeError", "load", "MoELayerW4", "ExpertGate", "ResidualNorm", "PagedKVCache"]

_HOMES = {"MoELayerW4": "layer", "ExpertGate": "gate", "ResidualNorm": "residual", "PagedKVCache": "kv"}


def __getattr__(name):
    if name in _HOMES:
        from importlib import import_module
        return getattr(import_module("." + _HOMES[name], __name__), name)
    raise AttributeError(name)
