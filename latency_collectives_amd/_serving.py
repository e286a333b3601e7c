"""Binding of the C ABI in ``include/ar_serving.h``: the 8-bit paged cache and its attention, the life of
a cache's pages, attention over packed prompts.

As in :mod:`latency_collectives_amd._decode`, every function has the name of the C entry point it wraps
and takes torch tensors; the calls are those of the compiled module ``_serving_calls``
(``csrc_serving/ar_serving_bind.cpp``), loaded with the library on first use. Nothing here computes, and
there is no fallback.

A request's life over caches of either width::

    ar_page_tables(...)                                          # pages for the step's tokens
    ar_kv8_norm_rope_append(h, q, k, v, ...)                     # every layer
    ar_kv8_attention(h, q_out, data, scales, table, kv_len, q_start, out)
    ar_pages_fork(src, dst, kv_len, table, shares, ...)          # sampled several ways
    ar_pages_copy([data, scales, ...], copy_src, copy_dst)       # every layer's cache
    ar_pages_free(requests, kv_len, table, shares, ...)          # done
    ar_pages_compact(kv_len, table, shares, ...)                 # now and then, and
    ar_pages_copy([data, scales, ...], move_src, move_dst)
"""

from __future__ import annotations

import ctypes
import struct

from . import _decode
from ._ar import ArError, ar_last_error, lib

# Every symbol include/ar_serving.h declares.
SERVING_EXPORTS = (
    "ar_kv8_create", "ar_kv8_destroy", "ar_kv8_append", "ar_kv8_read", "ar_kv8_norm_rope_append",
    "ar_kv8_attention", "ar_pages_fork", "ar_pages_free", "ar_pages_compact", "ar_pages_copy",
    "ar_prompt_create", "ar_prompt_destroy", "ar_prompt_attention",
)

# The calls of the compiled module.
_CALLS = tuple(n for n in SERVING_EXPORTS if not n.endswith(("_create", "_destroy")))

__all__ = ["SERVING_EXPORTS", "ar_kv8_create", "ar_kv8_destroy", "ar_kv8_cache", "ar_prompt_create",
           "ar_prompt_destroy", "ar_pages_scratch"]

# The argument structs of include/ar_serving.h, field for field (native alignment), beside those it
# shares with include/ar_decode.h.
_FORK = struct.Struct("@12P q 6i 0q")
_FREE = struct.Struct("@9P q 6i 0q")
_COMPACT = struct.Struct("@10P 2q 6i 0q")
_COPY = struct.Struct("@4P 3i 0q")
_PROMPT = struct.Struct("@6P 8q d 5i 0q")

_entry = None


def _bind():
    """The entry points; struct arguments go as packed bytes."""
    global _entry
    if _entry is None:
        L = lib()
        vp, i32 = ctypes.c_void_p, ctypes.c_int
        for name in SERVING_EXPORTS:
            fn = getattr(L, name)
            if name.endswith("_destroy"):
                fn.argtypes, fn.restype = [vp], None
            elif name == "ar_kv8_create":
                fn.argtypes, fn.restype = [i32, i32, i32], vp
            elif name == "ar_prompt_create":
                fn.argtypes, fn.restype = [i32, i32], vp
            elif name.startswith("ar_pages_"):
                fn.argtypes, fn.restype = [ctypes.c_char_p, vp], i32
            else:
                fn.argtypes, fn.restype = [vp, ctypes.c_char_p, vp], i32
        _entry = L
    return _entry


def _setup() -> None:
    """Loads the library and the compiled calls, which become attributes of this module."""
    _bind()
    import torch  # noqa: F401  (its libraries are what the compiled module links to)

    try:
        from . import _serving_calls
    except ImportError as e:
        raise ImportError(
            f"{e}; build it with `python -m latency_collectives_amd.build`") from e
    _serving_calls._setup(ArError)
    for name in _CALLS:
        globals()[name] = getattr(_serving_calls, name)


def __getattr__(name):
    if name in _CALLS:
        _setup()
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def _made(p, geometry):
    if not p:
        raise ArError(-1, ar_last_error())
    h = _decode._Handle(p)
    h.geometry = geometry
    import torch

    if torch.cuda.is_available():
        h.device = torch.cuda.current_device()
    return h


def ar_kv8_create(kv_heads: int, head_dim: int, page_size: int):
    """A handle for 8-bit caches of one geometry, whose attention runs on the GPU that is current now."""
    kv_heads, head_dim, page_size = int(kv_heads), int(head_dim), int(page_size)
    return _made(_bind().ar_kv8_create(kv_heads, head_dim, page_size), (kv_heads, head_dim, page_size, 8))


def ar_kv8_destroy(h) -> None:
    _bind().ar_kv8_destroy(h)
    h.value = None


def ar_kv8_cache(h, num_pages: int, device="cuda"):
    """(data, scales) of an empty cache of `num_pages` pages for one layer."""
    import torch

    heads, d, page, _ = h.geometry
    return (torch.zeros(num_pages, heads, 2, page * d, dtype=torch.uint8, device=device),
            torch.zeros(num_pages, heads, page // 16, 2, dtype=torch.uint8, device=device))


def ar_pages_scratch(num_pages: int, device="cuda"):
    """The scratch words of ar_pages_free and ar_pages_compact."""
    import torch

    return torch.zeros((num_pages + 31) // 32 + 1, dtype=torch.int32, device=device)


def ar_prompt_create(kv_heads: int, head_dim: int):
    """A handle for the attention over packed prompts, on the GPU that is current now."""
    kv_heads, head_dim = int(kv_heads), int(head_dim)
    return _made(_bind().ar_prompt_create(kv_heads, head_dim), (kv_heads, head_dim))


def ar_prompt_destroy(h) -> None:
    _bind().ar_prompt_destroy(h)
    h.value = None
