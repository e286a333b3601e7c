"""Sizes that the attention over the 4-bit cache refuses before anything is launched. No GPU is needed:
the calls end in their checks."""

import pytest

from tests.test_decode_host import A, D, _attn  # noqa: F401  (fixtures)


@pytest.mark.parametrize("heads,group,nreq,tokens", [
    (1024, 1, 180000, 180000),  # more jobs than units can be counted for: 12 of each job's are its start and end
    (1024, 1, 1 << 20, 1 << 20),
    (1024, 64, 1, 1 << 25),  # rows of a kv head past 31 bits
    (1, 65536, 1, 1 << 16),
    (1, 1, 1, 2 ** 31 - 1),
    (1, 65536, 1, 2 ** 31 - 1),
])
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("width", [0, 8, 2 ** 31 - 1])
def test_more_rows_than_the_split_can_count(D, A, heads, group, nreq, tokens, dtype, width):
    h = D.ar_kv4_create(heads, 64, 1024)
    hq, dim = heads * group, 64
    args = _attn(qt=hq * dim, qh=dim, ot=hq * dim, oh=dim, stride=width, width=width, dtype=dtype, ntokens=tokens,
                 hq=hq, nreq=nreq)
    assert D._entry.ar_kv4_attention(h, D._ATTENTION.pack(*args), None) == A.AR_ETOOBIG
    assert "rows" in A.ar_last_error()
    D.ar_kv4_destroy(h)


@pytest.mark.parametrize("scale", [3e38, -3e38, 1e39, 1e308])
def test_scales_past_binary32(D, A, scale):
    """In base-2 units, as the kernels hold it, such a scale would be an infinity, and NaN for a product
    that is zero."""
    h = D.ar_kv4_create(2, 128, 16)
    assert D._entry.ar_kv4_attention(h, D._ATTENTION.pack(*_attn(scale=scale)), None) == A.AR_EINVAL
    assert "scale" in A.ar_last_error()
    D.ar_kv4_destroy(h)
