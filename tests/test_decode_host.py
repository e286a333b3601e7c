"""Decode operators without a GPU: exports and struct layouts of include/ar_decode.h, refusals of
bad arguments before anything is launched, and the references the GPU tests compare with."""

import ctypes
import os
import re
import struct
import subprocess

import pytest
import torch

from tests import decode_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ar_decode.h")


@pytest.fixture(scope="module")
def D():
    from latency_collectives_amd import build

    build.ensure_built()
    from latency_collectives_amd import _decode

    _decode._setup()
    return _decode


@pytest.fixture(scope="module")
def A():
    from latency_collectives_amd import _ar

    return _ar


def _text():
    with open(HEADER) as f:
        return re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)


def test_every_declared_symbol_is_exported_and_bound(D):
    names = sorted(set(re.findall(r"\b(ar_[a-z0-9_]+)\s*\(", _text())))
    assert names == sorted(D.DECODE_EXPORTS)
    import latency_collectives_amd as lc

    for n in names:
        assert hasattr(D.lib(), n), n
        assert callable(getattr(lc, n)), n


def test_struct_layouts_match_the_header(D, tmp_path):
    """sizeof and the last field's offset of every argument struct, from the compiler."""
    src = tmp_path / "s.cpp"
    src.write_text(
        f'#include "{HEADER}"\n#include <cstddef>\n#include <cstdio>\nint main() {{\n'
        'printf("%zu %zu\\n", sizeof(ar_page_tables_args), offsetof(ar_page_tables_args, page_size));\n'
        'printf("%zu %zu\\n", sizeof(ar_qk_norm_rope_args), offsetof(ar_qk_norm_rope_args, interleaved));\n'
        'printf("%zu %zu\\n", sizeof(ar_kv4_rows_args), offsetof(ar_kv4_rows_args, ntokens));\n'
        'printf("%zu %zu\\n", sizeof(ar_kv4_attention_args), offsetof(ar_kv4_attention_args, window));\n}\n')
    exe = tmp_path / "s"
    subprocess.run(["g++", str(src), "-o", str(exe)], check=True)
    got = [tuple(map(int, x.split())) for x in
           subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()]
    mine = []
    for s in (D._PAGE_TABLES, D._NORM_ROPE, D._ROWS, D._ATTENTION):
        fmt = s.format.replace("0q", "").rstrip()
        mine.append((s.size, struct.calcsize(fmt) - 4))
    assert got == mine


# ------------------------------------------------------------------ refusals through the C ABI

PTR = 1 << 20  # an aligned address that is never used: every call here ends in its checks


def _tables(**kw):
    f = dict(cached=PTR, new=PTR, pool=PTR, free=PTR, table=PTR, kv=2 * PTR, q_start=PTR, slots=PTR,
             positions=PTR, pool_out=2 * PTR, refused=PTR, stride=8, nreq=4, width=8, nfree=16,
             ntokens=4, page=16)
    f.update(kw)
    return tuple(f.values())


def _rope(**kw):
    f = dict(q=PTR, k=PTR, v=PTR, q_out=2 * PTR, k_out=2 * PTR, positions=PTR, cos_sin=PTR, wq=PTR,
             wk=PTR, slots=PTR, data=PTR, scales=PTR, qt=1024, qh=128, kt=256, kh=128, vt=256, vh=128,
             ot=1024, oh=128, ct=256, ch=128, pages=4, eps=1e-6, dtype=1, ntokens=3, hq=8, hkv=2,
             d=128, rot=128, rows=64, inter=0)
    f.update(kw)
    return tuple(f.values())


def _rows(**kw):
    f = dict(k=PTR, v=PTR, slots=PTR, data=PTR, scales=PTR, kt=256, kh=128, vt=256, vh=128, pages=4,
             dtype=1, ntokens=3)
    f.update(kw)
    return tuple(f.values())


def _attn(**kw):
    f = dict(q=PTR, out=PTR, lse=0, data=PTR, scales=PTR, table=PTR, kv=PTR, q_start=PTR, qt=1024,
             qh=128, ot=1024, oh=128, stride=8, pages=4, scale=0.1, dtype=1, ntokens=3, hq=8, nreq=3,
             width=8, window=0)
    f.update(kw)
    return tuple(f.values())


@pytest.mark.parametrize("kw,code,word", [
    (dict(nreq=-1), "EINVAL", "negative"), (dict(ntokens=-1), "EINVAL", "negative"),
    (dict(nfree=-1), "EINVAL", "negative"), (dict(width=-1), "EINVAL", "negative"),
    (dict(nreq=4097), "ETOOBIG", "4096"), (dict(page=0), "EINVAL", "page_size"),
    (dict(stride=7), "EINVAL", "table_stride"), (dict(pool=0), "EINVAL", "null"),
    (dict(pool_out=0), "EINVAL", "null"), (dict(q_start=0), "EINVAL", "null"),
    (dict(cached=0), "EINVAL", "null"), (dict(new=0), "EINVAL", "null"),
    (dict(table=0), "EINVAL", "null"), (dict(kv=0), "EINVAL", "null"),
    (dict(refused=0), "EINVAL", "null"), (dict(slots=0), "EINVAL", "null"),
    (dict(positions=0), "EINVAL", "null"), (dict(free=0), "EINVAL", "null"),
    (dict(pool_out=PTR), "EINVAL", "must not be"), (dict(kv=PTR), "EINVAL", "must not be"),
])
def test_page_tables_refusals(D, A, kw, code, word):
    assert D._entry.ar_page_tables(D._PAGE_TABLES.pack(*_tables(**kw)), None) == getattr(A, "AR_" + code)
    assert word in A.ar_last_error()


def test_null_arguments_are_refused(D, A):
    assert D._entry.ar_page_tables(None, None) == A.AR_EINVAL
    assert D._entry.ar_qk_norm_rope(None, None) == A.AR_EINVAL
    for name, s, f in (("append", D._ROWS, _rows), ("read", D._ROWS, _rows),
                       ("norm_rope_append", D._NORM_ROPE, _rope), ("attention", D._ATTENTION, _attn)):
        fn = getattr(D._entry, "ar_kv4_" + name)
        assert fn(None, s.pack(*f()), None) == A.AR_EINVAL
        assert "handle" in A.ar_last_error()
    D._entry.ar_kv4_destroy(None)


_ROPE_BAD = [
    (dict(dtype=2), "ENOTSUP", "dtype"), (dict(ntokens=-1), "EINVAL", "negative"),
    (dict(hq=-1), "EINVAL", "negative"), (dict(hq=65537), "ETOOBIG", "heads"),
    (dict(rot=12), "EINVAL", "rot"), (dict(rot=136), "EINVAL", "rot"),
    (dict(eps=-1.0), "EINVAL", "eps"), (dict(eps=float("nan")), "EINVAL", "eps"),
    (dict(positions=0), "EINVAL", "rotation"), (dict(cos_sin=0), "EINVAL", "rotation"),
    (dict(rows=0), "EINVAL", "rotation"), (dict(cos_sin=PTR + 4), "EINVAL", "cos_sin"),
    (dict(wq=PTR + 2), "EINVAL", "weight"), (dict(q=0), "EINVAL", "null q"),
    (dict(q=PTR + 4), "EINVAL", "q:"), (dict(qt=1022), "EINVAL", "q:"), (dict(kh=-128), "EINVAL", "k:"),
    (dict(k=0), "EINVAL", "null k"), (dict(q_out=0), "EINVAL", "null q_out"),
    (dict(q_out=PTR, ot=2048), "EINVAL", "in place"), (dict(dtype=0, q=PTR + 8), "EINVAL", "q:"),
]


@pytest.mark.parametrize("kw,code,word", _ROPE_BAD + [
    (dict(d=4), "EINVAL", "head_dim"), (dict(d=132), "EINVAL", "head_dim"),
    (dict(d=264), "EINVAL", "head_dim"), (dict(k_out=0), "EINVAL", "null k_out"),
    (dict(k_out=PTR, ct=512), "EINVAL", "in place"),
])
def test_norm_rope_refusals(D, A, kw, code, word):
    assert D._entry.ar_qk_norm_rope(D._NORM_ROPE.pack(*_rope(**kw)), None) == getattr(A, "AR_" + code)
    assert word in A.ar_last_error()


@pytest.fixture()
def handle(D):
    h = D.ar_kv4_create(2, 128, 16)
    yield h
    D.ar_kv4_destroy(h)


@pytest.mark.parametrize("args,word", [
    ((0, 128, 16), "kv_heads"), ((1025, 128, 16), "kv_heads"), ((2, 80, 16), "head_dim"),
    ((2, 512, 16), "head_dim"), ((2, 128, 8), "page_size"), ((2, 128, 48), "page_size"),
    ((2, 128, 2048), "page_size"),
])
def test_create_refusals(D, args, word):
    with pytest.raises(D.ArError, match=word):
        D.ar_kv4_create(*args)


@pytest.mark.parametrize("kw,code,word", [
    (dict(dtype=2), "ENOTSUP", "dtype"), (dict(ntokens=-1), "EINVAL", "negative"),
    (dict(data=0), "EINVAL", "null cache"), (dict(scales=0), "EINVAL", "null cache"),
    (dict(data=PTR + 8), "EINVAL", "aligned"), (dict(pages=0), "EINVAL", "num_pages"),
    (dict(pages=1 << 31), "EINVAL", "num_pages"), (dict(slots=0), "EINVAL", "slots"),
    (dict(k=0), "EINVAL", "null k"), (dict(v=0), "EINVAL", "null v"),
    (dict(vt=258), "EINVAL", "v:"), (dict(k=PTR + 2), "EINVAL", "k:"),
])
@pytest.mark.parametrize("name", ["append", "read"])
def test_cache_row_refusals(D, A, handle, name, kw, code, word):
    fn = getattr(D._entry, "ar_kv4_" + name)
    assert fn(handle, D._ROWS.pack(*_rows(**kw)), None) == getattr(A, "AR_" + code)
    assert word in A.ar_last_error()


@pytest.mark.parametrize("kw,code,word", _ROPE_BAD + [
    (dict(d=64, rot=64), "EINVAL", "handle"), (dict(hkv=4), "EINVAL", "handle"),
    (dict(data=0), "EINVAL", "null cache"), (dict(pages=0), "EINVAL", "num_pages"),
    (dict(slots=0), "EINVAL", "slots"), (dict(v=0), "EINVAL", "null v"),
])
def test_norm_rope_append_refusals(D, A, handle, kw, code, word):
    rc = D._entry.ar_kv4_norm_rope_append(handle, D._NORM_ROPE.pack(*_rope(**kw)), None)
    assert rc == getattr(A, "AR_" + code)
    assert word in A.ar_last_error()


@pytest.mark.parametrize("kw,code,word", [
    (dict(dtype=2), "ENOTSUP", "dtype"), (dict(ntokens=-1), "EINVAL", "negative"),
    (dict(nreq=-1), "EINVAL", "negative"), (dict(width=-1), "EINVAL", "negative"),
    (dict(hq=0), "EINVAL", "q_heads"), (dict(hq=7), "EINVAL", "q_heads"),
    (dict(hq=131072), "ETOOBIG", "heads"), (dict(window=-1), "EINVAL", "window"),
    (dict(scale=float("inf")), "EINVAL", "scale"), (dict(scale=float("nan")), "EINVAL", "scale"),
    (dict(data=0), "EINVAL", "null cache"), (dict(scales=PTR + 1), "EINVAL", "aligned"),
    (dict(pages=0), "EINVAL", "num_pages"), (dict(stride=4), "EINVAL", "table_stride"),
    (dict(q=0), "EINVAL", "null q"), (dict(out=0), "EINVAL", "null q"),
    (dict(kv=0), "EINVAL", "null request"), (dict(q_start=0), "EINVAL", "null request"),
    (dict(table=0), "EINVAL", "null request"), (dict(q=PTR + 8), "EINVAL", "16 bytes"),
    (dict(qt=1028), "EINVAL", "16 bytes"), (dict(oh=132), "EINVAL", "16 bytes"),
    (dict(qt=-1024), "EINVAL", "negative"),
])
def test_attention_refusals(D, A, handle, kw, code, word):
    rc = D._entry.ar_kv4_attention(handle, D._ATTENTION.pack(*_attn(**kw)), None)
    assert rc == getattr(A, "AR_" + code)
    assert word in A.ar_last_error()


def test_empty_calls_launch_nothing(D, A, handle):
    assert D._entry.ar_kv4_attention(handle, D._ATTENTION.pack(*_attn(ntokens=0, q=0)), None) == A.AR_OK
    assert D._entry.ar_kv4_append(handle, D._ROWS.pack(*_rows(ntokens=0, k=0)), None) == A.AR_OK
    assert D._entry.ar_kv4_read(handle, D._ROWS.pack(*_rows(ntokens=0, k=0)), None) == A.AR_OK
    assert D._entry.ar_qk_norm_rope(D._NORM_ROPE.pack(*_rope(ntokens=0, q=0)), None) == A.AR_OK


def test_tensors_of_the_wrong_place_type_or_shape_are_refused(D, handle):
    x = torch.zeros(3, 2, 128)
    with pytest.raises(ValueError, match="GPU"):
        D.ar_qk_norm_rope(x, x, x, x)
    with pytest.raises(ValueError, match="dtype"):
        D.ar_qk_norm_rope(x.half(), x.half(), x.half(), x.half())
    with pytest.raises(ValueError, match="GPU"):
        D.ar_kv4_append(handle, x, x, torch.zeros(3, dtype=torch.int64), x, x)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="table"):
        D.ar_page_tables(i, i, i, i, i, i, i, i, i, i, i, 16)
    with pytest.raises(ValueError, match="head_dim"):
        D.ar_kv4_attention(handle, torch.zeros(3, 8, 64), x, x, i, i, i, x)


# ------------------------------------------------------------------ the references themselves


def test_quantiser_reference_on_known_values():
    x = torch.zeros(1, 32)
    x[0, :8] = torch.tensor([6.0, -6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 5.0])
    x[0, 8:11] = torch.tensor([3.5, -0.26, -0.0])
    code, scale = R.quantise(x)
    assert int(scale[0, 0]) == 127  # 6 = 6 * 2^0
    assert code[0, :11].tolist() == [7, 15, 0, 2, 2, 4, 4, 6, 6, 9, 8]
    code, scale = R.quantise(x * (1 + 2.0 ** -20))
    assert int(scale[0, 0]) == 128
    assert R.quantise(torch.zeros(1, 32))[1].item() == 1
    assert R.quantise(torch.full((1, 32), 3.4e38))[1].item() == 252
    y = torch.ones(1, 64)
    y[0, 40] = float("inf")
    assert R.quantise(y)[1].tolist() == [[125, 255]]


def test_page_table_reference_on_a_small_step():
    got = R.page_tables([3, 4, 0, 9], [1, 1, 6, -1], [1, 4], [50, 51, 52, 53], [[7, -1], [8, -1], [-1, -1], [9, 9]],
                        9, 4)
    table, kv, q_start, slots, positions, pool, refused = got
    assert table == [[7, -1], [8, 51], [52, 53], [9, 9]]
    assert kv == [4, 5, 6, 9] and q_start == [0, 1, 2, 8, 8]
    assert slots == [31, 204, 208, 209, 210, 211, 212, 213, -1]
    assert positions == [3, 4, 0, 1, 2, 3, 4, 5, -1]
    assert pool == [4, 4] and refused == [0, 0, 0, 1]
