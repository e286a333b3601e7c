"""Serving operators without a GPU: exports and struct layouts of include/ar_serving.h, refusals of bad
arguments before anything is launched, the compiled binding, and the references the GPU tests compare with."""

import ctypes
import os
import re
import struct
import subprocess

import pytest
import torch

from tests import serving_ref as S
from tests.test_decode_host import PTR, _attn, _rope, _rows
from tests.test_decode_host import _ROPE_BAD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ar_serving.h")


@pytest.fixture(scope="module")
def D():
    from latency_collectives_amd import build

    build.ensure_built()
    from latency_collectives_amd import _decode

    _decode._setup()
    return _decode


@pytest.fixture(scope="module")
def V():
    from latency_collectives_amd import build

    build.ensure_built()
    from latency_collectives_amd import _serving

    _serving._setup()
    return _serving


@pytest.fixture(scope="module")
def A():
    from latency_collectives_amd import _ar

    return _ar


@pytest.fixture()
def handle(V):
    h = V.ar_kv8_create(2, 128, 16)
    yield h
    V.ar_kv8_destroy(h)


def _text():
    with open(HEADER) as f:
        return re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)


def test_every_declared_symbol_is_exported_and_bound(V):
    names = sorted(set(re.findall(r"\b(ar_[a-z0-9_]+)\s*\(", _text())))
    assert names == sorted(V.SERVING_EXPORTS)
    import latency_collectives_amd as lc

    for n in names:
        assert hasattr(V.lib(), n), n
        assert getattr(lc, n).__name__ == n
    assert "scale=None" in lc.ar_kv8_attention.__text_signature__


def test_struct_layouts_match_the_header(V, tmp_path):
    """sizeof and the last field's offset of every argument struct, from the compiler."""
    src = tmp_path / "s.cpp"
    names = [("ar_pages_fork_args", "page_size", V._FORK), ("ar_pages_free_args", "page_size", V._FREE),
             ("ar_pages_compact_args", "page_size", V._COMPACT), ("ar_pages_copy_args", "num_pages", V._COPY),
             ("ar_prompt_attention_args", "window", V._PROMPT)]
    lines = "".join(f'printf("%zu %zu\\n", sizeof({n}), offsetof({n}, {f}));\n' for n, f, _ in names)
    src.write_text(f'#include "{HEADER}"\n#include <cstddef>\n#include <cstdio>\nint main() {{\n{lines}}}\n')
    exe = tmp_path / "s"
    subprocess.run(["g++", str(src), "-o", str(exe)], check=True)
    got = [tuple(map(int, x.split())) for x in
           subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()]
    assert got == [(s.size, struct.calcsize(s.format.replace("0q", "").rstrip()) - 4) for _, _, s in names]


# ------------------------------------------------------------------ refusals through the C ABI


def _fork(**kw):
    f = dict(src=PTR, dst=PTR, kv=PTR, table=PTR, shares=PTR, pool=PTR, free=PTR, kv_out=2 * PTR, pool_out=2 * PTR,
             copy_src=PTR, copy_dst=PTR, refused=PTR, stride=8, count=3, nreq=4, width=8, pages=32, nfree=32, page=16)
    f.update(kw)
    return tuple(f.values())


def _free(**kw):
    f = dict(requests=PTR, kv=PTR, table=PTR, shares=PTR, pool=PTR, free=PTR, kv_out=2 * PTR, pool_out=2 * PTR,
             scratch=PTR, stride=8, count=3, nreq=4, width=8, pages=32, nfree=32, page=16)
    f.update(kw)
    return tuple(f.values())


def _compact(**kw):
    f = dict(kv=PTR, table=PTR, shares=PTR, table_out=2 * PTR, shares_out=2 * PTR, free=PTR, pool_out=PTR,
             move_src=PTR, move_dst=PTR, scratch=PTR, stride=8, out_stride=8, nreq=4, width=8, pages=32, nfree=32,
             nmoves=16, page=16)
    f.update(kw)
    return tuple(f.values())


def _prompt(**kw):
    f = dict(q=PTR, k=PTR, v=PTR, out=PTR, lse=0, q_start=PTR, qt=1024, qh=128, kt=256, kh=128, vt=256, vh=128,
             ot=1024, oh=128, scale=0.1, dtype=1, ntokens=3, hq=8, nreq=2, window=0)
    f.update(kw)
    return tuple(f.values())


_PAGES_BAD = [
    (dict(nreq=-1), "EINVAL", "negative"), (dict(width=-1), "EINVAL", "negative"),
    (dict(nreq=4097), "ETOOBIG", "4096"), (dict(page=0), "EINVAL", "page_size"),
    (dict(stride=7), "EINVAL", "table_stride"), (dict(pages=0), "EINVAL", "num_pages"),
    (dict(shares=0), "EINVAL", "null"), (dict(pool_out=0), "EINVAL", "null"),
    (dict(kv=0), "EINVAL", "null request"), (dict(table=0), "EINVAL", "null request"),
]


@pytest.mark.parametrize("kw,code,word", _PAGES_BAD + [
    (dict(count=-1), "EINVAL", "negative"), (dict(count=4097), "ETOOBIG", "4096"),
    (dict(nfree=-1), "EINVAL", "negative"), (dict(pool=0), "EINVAL", "null"),
    (dict(src=0), "EINVAL", "null list"), (dict(dst=0), "EINVAL", "null list"),
    (dict(copy_src=0), "EINVAL", "null list"), (dict(copy_dst=0), "EINVAL", "null list"),
    (dict(refused=0), "EINVAL", "null list"), (dict(free=0), "EINVAL", "null free"),
    (dict(kv_out=0), "EINVAL", "null request"), (dict(kv_out=PTR), "EINVAL", "must not be"),
    (dict(pool_out=PTR), "EINVAL", "must not be"),
])
def test_fork_refusals(V, A, kw, code, word):
    assert V._entry.ar_pages_fork(V._FORK.pack(*_fork(**kw)), None) == getattr(A, "AR_" + code)
    assert word in A.ar_last_error()


@pytest.mark.parametrize("kw,code,word", _PAGES_BAD + [
    (dict(count=-1), "EINVAL", "negative"), (dict(count=4097), "ETOOBIG", "4096"),
    (dict(nfree=-1), "EINVAL", "negative"), (dict(pool=0), "EINVAL", "null"),
    (dict(requests=0), "EINVAL", "null list"), (dict(scratch=0), "EINVAL", "scratch"),
    (dict(pages=(1 << 19) + 1), "ETOOBIG", "pages"), (dict(free=0), "EINVAL", "null free"),
    (dict(kv_out=0), "EINVAL", "null request"), (dict(kv_out=PTR), "EINVAL", "must not be"),
    (dict(pool_out=PTR), "EINVAL", "must not be"),
])
def test_free_refusals(V, A, kw, code, word):
    assert V._entry.ar_pages_free(V._FREE.pack(*_free(**kw)), None) == getattr(A, "AR_" + code)
    assert word in A.ar_last_error()


@pytest.mark.parametrize("kw,code,word", _PAGES_BAD + [
    (dict(scratch=0), "EINVAL", "scratch"), (dict(shares_out=0), "EINVAL", "shares"),
    (dict(pages=(1 << 19) + 1, nfree=1 << 20, nmoves=1 << 20), "ETOOBIG", "pages"),
    (dict(nfree=31), "EINVAL", "free list"), (dict(nmoves=15), "EINVAL", "moves"),
    (dict(free=0), "EINVAL", "null"), (dict(move_src=0), "EINVAL", "null list"),
    (dict(move_dst=0), "EINVAL", "null list"), (dict(out_stride=7), "EINVAL", "out_stride"),
    (dict(table_out=0), "EINVAL", "null request"), (dict(table_out=PTR), "EINVAL", "must not be"),
    (dict(shares_out=PTR), "EINVAL", "must not be"),
])
def test_compact_refusals(V, A, kw, code, word):
    assert V._entry.ar_pages_compact(V._COMPACT.pack(*_compact(**kw)), None) == getattr(A, "AR_" + code)
    assert word in A.ar_last_error()


def _copy(V, buffers=(PTR, PTR), sizes=(64, 64), count=3, pages=4, src=PTR, dst=PTR, lists=True):
    n = len(buffers)
    b, s = (ctypes.c_void_p * n)(*buffers), (ctypes.c_int64 * n)(*sizes)
    at = (ctypes.addressof(b), ctypes.addressof(s)) if lists else (0, 0)
    return V._entry.ar_pages_copy(V._COPY.pack(*at, src, dst, n, count, pages), None)


def test_copy_refusals(V, A):
    assert _copy(V, count=-1) == A.AR_EINVAL and _copy(V, pages=-1) == A.AR_EINVAL
    assert _copy(V, src=0) == A.AR_EINVAL and _copy(V, dst=0) == A.AR_EINVAL and _copy(V, lists=False) == A.AR_EINVAL
    assert _copy(V, buffers=(PTR, 0)) == A.AR_EINVAL and "null buffer" in A.ar_last_error()
    assert _copy(V, sizes=(64, -1)) == A.AR_EINVAL
    assert _copy(V, sizes=(64, (1 << 29) + 1)) == A.AR_ETOOBIG
    assert _copy(V, count=0, src=0) == A.AR_OK and _copy(V, pages=0, src=0) == A.AR_OK
    assert _copy(V, buffers=(0, 0), sizes=(0, 0)) == A.AR_OK


def test_null_arguments_are_refused(V, D, A):
    for name in ("fork", "free", "compact", "copy"):
        assert getattr(V._entry, "ar_pages_" + name)(None, None) == A.AR_EINVAL
    for name, s, f in (("append", D._ROWS, _rows), ("read", D._ROWS, _rows),
                       ("norm_rope_append", D._NORM_ROPE, _rope), ("attention", D._ATTENTION, _attn)):
        assert getattr(V._entry, "ar_kv8_" + name)(None, s.pack(*f()), None) == A.AR_EINVAL
        assert "handle" in A.ar_last_error()
    assert V._entry.ar_prompt_attention(None, V._PROMPT.pack(*_prompt()), None) == A.AR_EINVAL
    assert "handle" in A.ar_last_error()
    V._entry.ar_kv8_destroy(None)
    V._entry.ar_prompt_destroy(None)


@pytest.mark.parametrize("args,word", [
    ((0, 128, 16), "kv_heads"), ((1025, 128, 16), "kv_heads"), ((2, 80, 16), "head_dim"),
    ((2, 512, 16), "head_dim"), ((2, 128, 8), "page_size"), ((2, 128, 48), "page_size"),
    ((2, 128, 2048), "page_size"),
])
def test_create_refusals(V, args, word):
    with pytest.raises(V.ArError, match=word):
        V.ar_kv8_create(*args)
    if word != "page_size":
        with pytest.raises(V.ArError, match=word):
            V.ar_prompt_create(*args[:2])


@pytest.mark.parametrize("kw,code,word", [
    (dict(dtype=2), "ENOTSUP", "dtype"), (dict(ntokens=-1), "EINVAL", "negative"),
    (dict(data=0), "EINVAL", "null cache"), (dict(scales=0), "EINVAL", "null cache"),
    (dict(data=PTR + 8), "EINVAL", "aligned"), (dict(pages=0), "EINVAL", "num_pages"),
    (dict(pages=1 << 31), "EINVAL", "num_pages"), (dict(slots=0), "EINVAL", "slots"),
    (dict(k=0), "EINVAL", "null k"), (dict(v=0), "EINVAL", "null v"),
    (dict(vt=258), "EINVAL", "v:"), (dict(k=PTR + 2), "EINVAL", "k:"),
])
@pytest.mark.parametrize("name", ["append", "read"])
def test_cache_row_refusals(V, D, A, handle, name, kw, code, word):
    fn = getattr(V._entry, "ar_kv8_" + name)
    assert fn(handle, D._ROWS.pack(*_rows(**kw)), None) == getattr(A, "AR_" + code)
    assert word in A.ar_last_error()


@pytest.mark.parametrize("kw,code,word", _ROPE_BAD + [
    (dict(d=64, rot=64), "EINVAL", "handle"), (dict(hkv=4), "EINVAL", "handle"),
    (dict(data=0), "EINVAL", "null cache"), (dict(pages=0), "EINVAL", "num_pages"),
    (dict(slots=0), "EINVAL", "slots"), (dict(v=0), "EINVAL", "null v"),
])
def test_norm_rope_append_refusals(V, D, A, handle, kw, code, word):
    rc = V._entry.ar_kv8_norm_rope_append(handle, D._NORM_ROPE.pack(*_rope(**kw)), None)
    assert rc == getattr(A, "AR_" + code)
    assert word in A.ar_last_error()


@pytest.mark.parametrize("kw,code,word", [
    (dict(dtype=2), "ENOTSUP", "dtype"), (dict(ntokens=-1), "EINVAL", "negative"),
    (dict(hq=7), "EINVAL", "q_heads"), (dict(window=-1), "EINVAL", "window"),
    (dict(scale=float("nan")), "EINVAL", "scale"), (dict(scale=3e38), "EINVAL", "scale"),
    (dict(data=0), "EINVAL", "null cache"), (dict(stride=4), "EINVAL", "table_stride"),
    (dict(q=0), "EINVAL", "null q"), (dict(kv=0), "EINVAL", "null request"),
    (dict(q=PTR + 8), "EINVAL", "16 bytes"), (dict(qt=-1024), "EINVAL", "negative"),
])
def test_attention_refusals(V, D, A, handle, kw, code, word):
    rc = V._entry.ar_kv8_attention(handle, D._ATTENTION.pack(*_attn(**kw)), None)
    assert rc == getattr(A, "AR_" + code)
    assert word in A.ar_last_error()


@pytest.mark.parametrize("kw,code,word", [
    (dict(dtype=2), "ENOTSUP", "dtype"), (dict(ntokens=-1), "EINVAL", "negative"),
    (dict(nreq=-1), "EINVAL", "negative"), (dict(hq=0), "EINVAL", "q_heads"), (dict(hq=7), "EINVAL", "q_heads"),
    (dict(hq=131072), "ETOOBIG", "heads"), (dict(window=-1), "EINVAL", "window"),
    (dict(scale=float("inf")), "EINVAL", "scale"), (dict(scale=-3e38), "EINVAL", "scale"),
    (dict(q=0), "EINVAL", "null q"), (dict(k=0), "EINVAL", "null q"), (dict(v=0), "EINVAL", "null q"),
    (dict(out=0), "EINVAL", "null q"), (dict(q_start=0), "EINVAL", "null q_start"),
    (dict(k=PTR + 8), "EINVAL", "16 bytes"), (dict(v=PTR + 8), "EINVAL", "16 bytes"),
    (dict(kt=260), "EINVAL", "16 bytes"), (dict(vh=132), "EINVAL", "16 bytes"), (dict(oh=132), "EINVAL", "16 bytes"),
    (dict(vt=-256), "EINVAL", "negative"), (dict(kt=1 << 23), "ETOOBIG", "apart"),
    (dict(dtype=0, vt=(1 << 21) + 4), "ETOOBIG", "apart"),
    (dict(ntokens=1 << 30), "ETOOBIG", "rows"), (dict(ntokens=2 ** 31 - 1, hq=2), "ETOOBIG", "rows"),
    (dict(ntokens=1 << 29, hq=2, nreq=1 << 29), "ETOOBIG", "rows"),
])
def test_prompt_refusals(V, A, kw, code, word):
    h = V.ar_prompt_create(2, 128)
    assert V._entry.ar_prompt_attention(h, V._PROMPT.pack(*_prompt(**kw)), None) == getattr(A, "AR_" + code)
    assert word in A.ar_last_error()
    V.ar_prompt_destroy(h)


def test_empty_calls_launch_nothing(V, D, A, handle):
    assert V._entry.ar_kv8_attention(handle, D._ATTENTION.pack(*_attn(ntokens=0, q=0)), None) == A.AR_OK
    assert V._entry.ar_kv8_append(handle, D._ROWS.pack(*_rows(ntokens=0, k=0)), None) == A.AR_OK
    assert V._entry.ar_kv8_read(handle, D._ROWS.pack(*_rows(ntokens=0, k=0)), None) == A.AR_OK
    h = V.ar_prompt_create(2, 128)
    assert V._entry.ar_prompt_attention(h, V._PROMPT.pack(*_prompt(ntokens=0, q=0)), None) == A.AR_OK
    assert V._entry.ar_prompt_attention(h, V._PROMPT.pack(*_prompt(nreq=0, q=0)), None) == A.AR_OK
    V.ar_prompt_destroy(h)


# ------------------------------------------------------------------ the compiled binding

X = torch.zeros(3, 2, 128)
I = torch.zeros(4, dtype=torch.int32)


def test_handles_of_another_kind_are_refused(V, D, handle):
    four, prompt = D.ar_kv4_create(2, 128, 16), V.ar_prompt_create(2, 128)
    for bad in (None, 3, object(), four, prompt):
        with pytest.raises(ValueError, match="h: needs a handle of ar_kv8_create"):
            V.ar_kv8_append(bad, X, X, I, X, X)
        with pytest.raises(ValueError, match="h: needs a handle of ar_kv8_create"):
            V.ar_kv8_attention(bad, X, X, X, I, I, I, X)
    for bad in (None, four, handle):
        with pytest.raises(ValueError, match="h: needs a handle of ar_prompt_create"):
            V.ar_prompt_attention(bad, X, X, X, I, X)
    for bad in (handle, prompt):
        with pytest.raises(ValueError, match="h: needs a handle of ar_kv4_create"):
            D.ar_kv4_append(bad, X, X, I, X, X)
    D.ar_kv4_destroy(four)
    V.ar_prompt_destroy(prompt)


def test_destroyed_handles_are_refused(V):
    h = V.ar_prompt_create(2, 128)
    V.ar_prompt_destroy(h)
    V.ar_prompt_destroy(h)  # as destroying nothing
    with pytest.raises((ValueError, V.ArError)):
        V.ar_prompt_attention(h, X, X, X, I, X)
    h = V.ar_kv8_create(2, 128, 16)
    V.ar_kv8_destroy(h)
    V.ar_kv8_destroy(h)
    with pytest.raises((ValueError, V.ArError)):
        V.ar_kv8_append(h, X, X, I, X, X)


def test_tensors_of_the_wrong_place_type_or_shape_are_refused(V, handle):
    with pytest.raises(ValueError, match="GPU"):
        V.ar_kv8_append(handle, X, X, torch.zeros(3, dtype=torch.int64), X, X)
    with pytest.raises(ValueError, match="head_dim 128, got 64"):
        V.ar_kv8_attention(handle, X[..., :64], X, X, I, I, I, X)
    with pytest.raises(ValueError, match="table"):
        V.ar_kv8_attention(handle, X, X, X, I, I, I, X)
    h = V.ar_prompt_create(2, 128)
    for bad in (X.half(), X.double()):
        with pytest.raises(ValueError, match="dtype"):
            V.ar_prompt_attention(h, bad, X, X, I, X)
    with pytest.raises(ValueError, match="head_dim 128, got 64"):
        V.ar_prompt_attention(h, X[..., :64], X, X, I, X)
    V.ar_prompt_destroy(h)
    with pytest.raises(ValueError, match="table"):
        V.ar_pages_fork(*[I] * 12, 16)
    with pytest.raises(ValueError, match="table"):
        V.ar_pages_free(*[I] * 9, 16)
    with pytest.raises(ValueError, match="table"):
        V.ar_pages_compact(*[I] * 10, 16)
    for bad in (None, X, 3, "x"):
        with pytest.raises(ValueError, match="buffers"):
            V.ar_pages_copy(bad, I, I)
    with pytest.raises(ValueError, match="buffers"):
        V.ar_pages_copy([3], I, I)


# ------------------------------------------------------------------ the references themselves


def test_codes_are_those_of_e4m3():
    code = torch.arange(256, dtype=torch.uint8)
    want = code.view(torch.float8_e4m3fn).double()
    assert torch.equal(S.E4M3.nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))
    y = torch.linspace(-500, 500, 4001, dtype=torch.float64)
    want = y.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
    assert torch.equal(S.rounded(y, 0), want)
    assert torch.equal(S.rounded(y * 2.0 ** -30, -30), want * 2.0 ** -30)
    tiny = torch.arange(-40, 41).double() * 2.0 ** -12
    assert torch.equal(S.rounded(tiny, 0), tiny.float().to(torch.float8_e4m3fn).double())


def test_scales_of_the_reference():
    assert S.exponent(448.0) == 0 and S.exponent(448.1) == 1 and S.exponent(224.0) == -1
    assert S.exponent(0.0) == -100 and S.exponent(1e-40) == -100 and S.exponent(3.4e38) == 119


def test_appending_reference_keeps_and_raises_scales():
    c = S.Cache(1, 1, 32, 32)
    one = torch.ones(1, 1, 32)
    c.append(one * 448, one, [0])
    assert c.e[0, 0, 0].tolist() == [0, -8]
    c.append(one, one * 1000, [1])
    assert c.e[0, 0, 0].tolist() == [0, 2]
    assert float(c.values[0, 0, 1, 0, 0]) == 1.0 and float(c.values[0, 0, 1, 1, 0]) == 1024.0
    c.append(one * 2.0 ** 20, one, [2, ])
    assert c.e[0, 0, 0].tolist() == [12, 2]
    assert float(c.values[0, 0, 0, 1, 0]) == 0.0  # 1 is nothing beside 2^20
    c.append(one, one, [0])
    assert c.e[0, 0, 0].tolist() == [-8, -8]


def test_page_references_on_a_small_pool():
    table = [[5, 6, 7], [-1, -1, -1], [2, -1, -1], [-1, -1, -1]]
    shares = [0] * 8
    t, shares, kv, pool, src, dst, refused = S.fork([0, 2, 0], [1, 3, 1], [10, 0, 4, 0], table, shares, [6, 8],
                                                    [9] * 6 + [3, 4], 4)
    assert t == [[5, 6, 7], [5, 6, 3], [2, -1, -1], [2, -1, -1]] and kv == [10, 10, 4, 4]
    assert shares == [0, 0, 1, 0, 0, 1, 1, 0] and pool == [7, 8]
    assert src == [7, -1, -1] and dst == [3, -1, -1] and refused == [0, 0, 1]
    shares, free, kv, pool = S.free_pages([0, 3, 0, 9], kv, t, shares, pool, [9] * 6 + [3, 4], 4)
    assert shares == [0] * 8 and kv == [0, 10, 4, 0] and pool == [6, 8] and free == [9] * 6 + [7, 4]
    t, shares, pool, src, dst = S.compact(kv, t, shares, 4, 4)
    assert pool == [4, 8] and src == [5, 6, -1, -1] and dst == [0, 1, -1, -1]
    assert t == [[-1] * 3, [0, 1, 3], [2, -1, -1], [-1] * 3]


@pytest.mark.parametrize("nreq", [2 ** 31 - 1, 2 ** 31 - 128])
def test_more_requests_than_are_counted(V, D, A, handle, nreq):
    """The lanes' places past the last request are counted in 31 bits too."""
    h = V.ar_prompt_create(2, 128)
    assert V._entry.ar_prompt_attention(h, V._PROMPT.pack(*_prompt(nreq=nreq)), None) == A.AR_ETOOBIG
    assert "requests" in A.ar_last_error()
    V.ar_prompt_destroy(h)
    assert V._entry.ar_kv8_attention(handle, D._ATTENTION.pack(*_attn(nreq=nreq)), None) == A.AR_ETOOBIG
    assert "requests" in A.ar_last_error()
