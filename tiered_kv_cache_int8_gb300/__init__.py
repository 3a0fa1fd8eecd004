"""Two-level KV cache for top-k sparse-attention decode on one GB300 (sm_103a), and
beside it rotary positions and a paged KV cache that stays in HBM.

The path (indexer + top-k, RESOLVE, attention, append) is CUDA in libhs.so,
reached through the C ABI in include/hs.h; ``hs`` is its ctypes binding, ``paged``
that of the rotary and paged-cache entry points.
"""
from .hs import HiSparseCache, HsError, lib  # noqa: F401


def __getattr__(name):   # paged imports torch: only when asked for
    if name in ("Rotary", "PagedKVCache"):
        from . import paged
        return getattr(paged, name)
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
