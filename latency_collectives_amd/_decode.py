"""ctypes binding of the C ABI in ``include/ar_decode.h``: the decode operators.

Every function has the name of the C entry point it wraps and takes torch tensors; sizes, types
and strides are the tensors' own. It checks what the C entry point cannot see (that tensors are on
the GPU, of the right type and shape) and raises ``ValueError``; a failing call raises
:class:`ArError` as in :mod:`latency_collectives_amd._ar`. Nothing here computes.

One step of tensor-parallel decoding on a rank, before its AllReduce::

    ar_page_tables(cached, new, pool, free_pages, table, kv_len, q_start, slots, positions,
                   pool_out, refused, page_size)                       # once a step
    for each layer:
        ar_kv4_norm_rope_append(h, q, k, v, q_out, positions, cos_sin, slots, data, scales, wq, wk)
        ar_kv4_attention(h, q_out, data, scales, table, kv_len, q_start, out)
"""

from __future__ import annotations

import ctypes
import math
import struct

from ._ar import AR_BFLOAT16, AR_FLOAT32, ArError, ar_last_error, lib

# Every symbol include/ar_decode.h declares.
DECODE_EXPORTS = (
    "ar_page_tables", "ar_qk_norm_rope", "ar_kv4_create", "ar_kv4_destroy", "ar_kv4_append",
    "ar_kv4_read", "ar_kv4_norm_rope_append", "ar_kv4_attention",
)

__all__ = [*DECODE_EXPORTS, "DECODE_EXPORTS", "ar_kv4_cache"]

# The argument structs of include/ar_decode.h, field for field (native alignment).
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


def _torch():
    import torch

    return torch


_types: dict = {}
_i32 = _i64 = _u8 = _f32 = None
_raw_stream = None


def _setup() -> None:
    global _i32, _i64, _u8, _f32, _raw_stream
    torch = _torch()
    _bind()
    _types.update({torch.bfloat16: AR_BFLOAT16, torch.float32: AR_FLOAT32})
    _i32, _i64, _u8, _f32 = torch.int32, torch.int64, torch.uint8, torch.float32
    # the current stream's handle without the Stream object that torch.cuda.current_stream() makes
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda d: torch.cuda.current_stream(d).cuda_stream)


def _ok(rc: int) -> None:
    if rc != 0:
        raise ArError(rc, ar_last_error())


def _stream(s, like) -> int:
    if s is None:
        return _raw_stream(like.get_device())
    return s if isinstance(s, int) else int(s.cuda_stream)


def _bad(name, why):
    raise ValueError(f"{name}: {why}")


def _vec(name, x, dtype, n):
    """A contiguous vector of at least n elements on the GPU; its address."""
    if not x.is_cuda:
        _bad(name, "not on the GPU")
    if x.dtype != dtype or not x.is_contiguous() or x.numel() < n:
        _bad(name, f"needs {n} contiguous elements of {dtype}")
    return x.data_ptr()


def _heads(name, x, dtype, tokens=None, heads=None, dim=None):
    """A [tokens, heads, dim] tensor with a contiguous last dimension: address, strides."""
    if not x.is_cuda:
        _bad(name, "not on the GPU")
    if x.dtype != dtype or x.dim() != 3:
        _bad(name, f"needs [tokens, heads, head_dim] of {dtype}")
    st = x.stride()
    sh = x.shape
    if st[2] != 1 and sh[2] != 1:
        _bad(name, "its last dimension is not contiguous")
    if tokens is not None and (sh[0] != tokens or sh[1] != heads or sh[2] != dim):
        _bad(name, f"needs [{tokens}, {heads}, {dim}], got {list(sh)}")
    return x.data_ptr(), st[0], st[1]


def _type(x):
    t = _types.get(x.dtype)
    if t is None:
        _bad("dtype", f"torch.bfloat16 or torch.float32, got {x.dtype}")
    return t


def _cache(h, data, scales):
    if not data.is_cuda or not scales.is_cuda:
        _bad("cache", "not on the GPU")
    heads, d, page = h.geometry
    n = data.shape[0]
    if data.dtype != _u8 or scales.dtype != _u8 or not data.is_contiguous() or not scales.is_contiguous():
        _bad("cache", "needs contiguous uint8 tensors")
    if data.numel() != n * heads * page * d or scales.numel() != n * heads * 2 * page * (d // 32):
        _bad("cache", f"data [pages, {heads}, 2, {page * d // 2}] and scales [pages, {heads}, 2, "
                      f"{d // 32}, {page}] are wanted, got {list(data.shape)} and {list(scales.shape)}")
    return data.data_ptr(), scales.data_ptr(), n


class _Handle(ctypes.c_void_p):
    """An ar_kv4 handle with its geometry (kv_heads, head_dim, page_size)."""

    geometry = (0, 0, 0)


def ar_page_tables(cached_len, new_len, pool, free_pages, table, kv_len, q_start, slots, positions,
                   pool_out, refused, page_size: int, stream=None) -> None:
    if _entry is None:
        _setup()
    n = cached_len.numel()
    t = slots.numel()
    if table.dim() != 2 or table.dtype != _i32 or not table.is_cuda or table.shape[0] < n or (
            table.shape[1] > 1 and table.stride(1) != 1):
        _bad("table", f"needs an int32 [{n}, pages] tensor on the GPU with contiguous rows")
    a = _PAGE_TABLES.pack(
        _vec("cached_len", cached_len, _i32, n), _vec("new_len", new_len, _i32, n),
        _vec("pool", pool, _i32, 2), _vec("free_pages", free_pages, _i32, 0), table.data_ptr(),
        _vec("kv_len", kv_len, _i32, n), _vec("q_start", q_start, _i32, n + 1),
        _vec("slots", slots, _i64, 0), _vec("positions", positions, _i32, t),
        _vec("pool_out", pool_out, _i32, 2), _vec("refused", refused, _i32, n),
        table.stride(0) if table.shape[0] > 1 else table.shape[1], n, table.shape[1],
        free_pages.numel(), t, page_size)
    _ok(_entry.ar_page_tables(a, _stream(stream, pool)))


def _norm_rope(q, k, v, q_out, k_out, positions, cos_sin, q_weight, k_weight, eps, interleaved,
               slots=0, data=0, scales=0, pages=0):
    dtype = q.dtype
    kind = _type(q)
    t, hq, d = q.shape
    hkv = k.shape[1]
    rot = rows = cs = pos = 0
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            _bad("cos_sin", "needs [rows, rot]")
        rows, rot = cos_sin.shape
        cs = _vec("cos_sin", cos_sin, _f32, 0)
    if positions is not None:
        pos = _vec("positions", positions, _i32, t)
    elif rot:
        _bad("positions", "a rotation needs them")
    wq = 0 if q_weight is None else _vec("q_weight", q_weight, dtype, d)
    wk = 0 if k_weight is None else _vec("k_weight", k_weight, dtype, d)
    qp, qt, qh = _heads("q", q, dtype)
    kp, kt, kh = _heads("k", k, dtype, t, hkv, d)
    op, ot, oh = _heads("q_out", q_out, dtype, t, hq, d)
    vp, vt, vh = (0, 0, 0) if v is None else _heads("v", v, dtype, t, hkv, d)
    cp, ct, ch = (0, 0, 0) if k_out is None else _heads("k_out", k_out, dtype, t, hkv, d)
    return _NORM_ROPE.pack(qp, kp, vp, op, cp, pos, cs, wq, wk, slots, data, scales, qt, qh, kt, kh,
                           vt, vh, ot, oh, ct, ch, pages, eps, kind, t, hq, hkv, d, rot, rows,
                           1 if interleaved else 0)


def ar_qk_norm_rope(q, k, q_out, k_out, positions=None, cos_sin=None, q_weight=None, k_weight=None,
                    eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    if _entry is None:
        _setup()
    a = _norm_rope(q, k, None, q_out, k_out, positions, cos_sin, q_weight, k_weight, eps, interleaved)
    _ok(_entry.ar_qk_norm_rope(a, _stream(stream, q)))


def ar_kv4_create(kv_heads: int, head_dim: int, page_size: int) -> _Handle:
    if _entry is None:
        _setup()
    p = _entry.ar_kv4_create(int(kv_heads), int(head_dim), int(page_size))
    if not p:
        raise ArError(-1, ar_last_error())
    h = _Handle(p)
    h.geometry = (int(kv_heads), int(head_dim), int(page_size))
    return h


def ar_kv4_destroy(h: _Handle) -> None:
    _bind().ar_kv4_destroy(h)
    h.value = None


def ar_kv4_cache(h: _Handle, num_pages: int, device="cuda"):
    """(data, scales) of an empty cache of `num_pages` pages for one layer."""
    heads, d, page = h.geometry
    torch = _torch()
    return (torch.zeros(num_pages, heads, 2, page * d // 2, dtype=torch.uint8, device=device),
            torch.zeros(num_pages, heads, 2, d // 32, page, dtype=torch.uint8, device=device))


def _rows(h, k, v, slots, data, scales):
    heads, d, _ = h.geometry
    t = k.shape[0]
    kp, kt, kh = _heads("k", k, k.dtype, t, heads, d)
    vp, vt, vh = _heads("v", v, k.dtype, t, heads, d)
    dp, sp, pages = _cache(h, data, scales)
    return _ROWS.pack(kp, vp, _vec("slots", slots, _i64, t), dp, sp, kt, kh, vt, vh, pages, _type(k), t)


def ar_kv4_append(h: _Handle, k, v, slots, data, scales, stream=None) -> None:
    _ok(_entry.ar_kv4_append(h, _rows(h, k, v, slots, data, scales), _stream(stream, k)))


def ar_kv4_read(h: _Handle, slots, data, scales, k, v, stream=None) -> None:
    _ok(_entry.ar_kv4_read(h, _rows(h, k, v, slots, data, scales), _stream(stream, k)))


def ar_kv4_norm_rope_append(h: _Handle, q, k, v, q_out, positions, cos_sin, slots, data, scales,
                            q_weight=None, k_weight=None, eps: float = 1e-6,
                            interleaved: bool = False, stream=None) -> None:
    dp, sp, pages = _cache(h, data, scales)
    a = _norm_rope(q, k, v, q_out, None, positions, cos_sin, q_weight, k_weight, eps, interleaved,
                   _vec("slots", slots, _i64, q.shape[0]), dp, sp, pages)
    _ok(_entry.ar_kv4_norm_rope_append(h, a, _stream(stream, q)))


def ar_kv4_attention(h: _Handle, q, data, scales, table, kv_len, q_start, out, lse=None,
                     scale: float | None = None, window: int = 0, stream=None) -> None:
    dtype = q.dtype
    kind = _type(q)
    t, hq, d = q.shape
    if d != h.geometry[1]:
        _bad("q", f"the handle is for head_dim {h.geometry[1]}, got {d}")
    n = kv_len.numel()
    if table.dim() != 2 or table.dtype != _i32 or not table.is_cuda or table.shape[0] < n or (
            table.shape[1] > 1 and table.stride(1) != 1):
        _bad("table", f"needs an int32 [{n}, pages] tensor on the GPU with contiguous rows")
    qp, qt, qh = _heads("q", q, dtype)
    op, ot, oh = _heads("out", out, dtype, t, hq, d)
    dp, sp, pages = _cache(h, data, scales)
    width = table.shape[1]
    a = _ATTENTION.pack(
        qp, op, 0 if lse is None else _vec("lse", lse, _f32, t * hq), dp, sp, table.data_ptr(),
        _vec("kv_len", kv_len, _i32, n), _vec("q_start", q_start, _i32, n + 1), qt, qh, ot, oh,
        table.stride(0) if table.shape[0] > 1 else width, pages,
        1.0 / math.sqrt(d) if scale is None else scale, kind, t, hq, n, width, window)
    _ok(_entry.ar_kv4_attention(h, a, _stream(stream, q)))
