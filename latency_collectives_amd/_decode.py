"""Binding of the C ABI in ``include/ar_decode.h``: the decode operators.

Every function has the name of the C entry point it wraps and takes torch tensors; sizes, types
and strides are the tensors' own. The calls are those of the compiled module ``_decode_calls``
(``csrc_decode/ar_decode_bind.cpp``), loaded with the library on first use: it checks what the C
entry point cannot see (that tensors are on the GPU, of the right type and shape, and that no
gradient is wanted of them) and raises ``ValueError``; a failing call raises :class:`ArError` as in
:mod:`latency_collectives_amd._ar`.
Nothing here computes, and there is no fallback.

One step of tensor-parallel decoding on a rank, before its AllReduce::

    ar_page_tables(cached, new, pool, free_pages, table, kv_len, q_start, slots, positions,
                   pool_out, refused, page_size)                       # once a step
    for each layer:
        ar_kv4_norm_rope_append(h, q, k, v, q_out, positions, cos_sin, slots, data, scales, wq, wk)
        ar_kv4_attention(h, q_out, data, scales, table, kv_len, q_start, out)
"""

from __future__ import annotations

import ctypes
import struct

from ._ar import ArError, ar_last_error, lib

# Every symbol include/ar_decode.h declares.
DECODE_EXPORTS = (
    "ar_page_tables", "ar_qk_norm_rope", "ar_kv4_create", "ar_kv4_destroy", "ar_kv4_append",
    "ar_kv4_read", "ar_kv4_norm_rope_append", "ar_kv4_attention",
)

# The calls of the compiled module.
_CALLS = ("ar_page_tables", "ar_qk_norm_rope", "ar_kv4_append", "ar_kv4_read",
          "ar_kv4_norm_rope_append", "ar_kv4_attention")

__all__ = ["DECODE_EXPORTS", "ar_kv4_create", "ar_kv4_destroy", "ar_kv4_cache"]

# The argument structs of include/ar_decode.h, field for field (native alignment): what a caller
# without tensors passes to the C entry points.
_PAGE_TABLES = struct.Struct("@11P q 5i 0q")
_NORM_ROPE = struct.Struct("@12P 11q d 8i")
_ROWS = struct.Struct("@5P 3q 2q 2i")
_ATTENTION = struct.Struct("@8P 6q d 6i")

_entry = None


def _bind():
    """The entry points; struct arguments go as packed bytes."""
    global _entry
    if _entry is None:
        L = lib()
        vp, i32 = ctypes.c_void_p, ctypes.c_int
        for name, args, res in (
            ("ar_page_tables", [ctypes.c_char_p, vp], i32),
            ("ar_qk_norm_rope", [ctypes.c_char_p, vp], i32),
            ("ar_kv4_create", [i32, i32, i32], vp),
            ("ar_kv4_destroy", [vp], None),
            ("ar_kv4_append", [vp, ctypes.c_char_p, vp], i32),
            ("ar_kv4_read", [vp, ctypes.c_char_p, vp], i32),
            ("ar_kv4_norm_rope_append", [vp, ctypes.c_char_p, vp], i32),
            ("ar_kv4_attention", [vp, ctypes.c_char_p, vp], i32),
        ):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _entry = L
    return _entry


def _setup() -> None:
    """Loads the library and the compiled calls, which become attributes of this module."""
    _bind()
    import torch  # noqa: F401  (its libraries are what the compiled module links to)

    try:
        from . import _decode_calls
    except ImportError as e:
        raise ImportError(
            f"{e}; build it with `python -m latency_collectives_amd.build`") from e
    _decode_calls._setup(ArError)
    for name in _CALLS:
        globals()[name] = getattr(_decode_calls, name)


def __getattr__(name):
    if name in _CALLS:
        _setup()
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


class _Handle(ctypes.c_void_p):
    """An ar_kv4 handle with its geometry (kv_heads, head_dim, page_size) and its GPU (-1: none)."""

    geometry = (0, 0, 0)
    device = -1


def ar_kv4_create(kv_heads: int, head_dim: int, page_size: int) -> _Handle:
    """A handle for caches of one geometry, whose attention runs on the GPU that is current now."""
    p = _bind().ar_kv4_create(int(kv_heads), int(head_dim), int(page_size))
    if not p:
        raise ArError(-1, ar_last_error())
    h = _Handle(p)
    h.geometry = (int(kv_heads), int(head_dim), int(page_size))
    import torch

    if torch.cuda.is_available():
        h.device = torch.cuda.current_device()
    return h


def ar_kv4_destroy(h: _Handle) -> None:
    _bind().ar_kv4_destroy(h)
    h.value = None


def ar_kv4_cache(h: _Handle, num_pages: int, device="cuda"):
    """(data, scales) of an empty cache of `num_pages` pages for one layer."""
    import torch

    heads, d, page = h.geometry
    return (torch.zeros(num_pages, heads, 2, page * d // 2, dtype=torch.uint8, device=device),
            torch.zeros(num_pages, heads, 2, d // 32, page, dtype=torch.uint8, device=device))
