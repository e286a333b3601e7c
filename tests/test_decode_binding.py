"""The compiled binding of the decode operators without a GPU: how it takes its arguments, and that
whatever it is given ends in a Python exception."""

import pytest
import torch


@pytest.fixture(scope="module")
def lc():
    from latency_collectives_amd import build

    build.ensure_built()
    import latency_collectives_amd as lc

    return lc


@pytest.fixture()
def handle(lc):
    h = lc.ar_kv4_create(2, 128, 16)
    yield h
    lc.ar_kv4_destroy(h)


X = torch.zeros(3, 2, 128)
I = torch.zeros(4, dtype=torch.int32)


def test_arguments_by_position_and_by_name(lc):
    with pytest.raises(TypeError, match="misses the argument 'q_out'"):
        lc.ar_qk_norm_rope(X, X)
    with pytest.raises(TypeError, match="at most 11 arguments"):
        lc.ar_qk_norm_rope(*[X] * 12)
    with pytest.raises(TypeError, match="unexpected argument 'epsilon'"):
        lc.ar_qk_norm_rope(X, X, X, X, epsilon=1.0)
    with pytest.raises(TypeError, match="multiple values for argument 'q'"):
        lc.ar_qk_norm_rope(X, X, X, X, q=X)
    # both orders reach the same check
    for call in (lambda: lc.ar_qk_norm_rope(X, X, X, X), lambda: lc.ar_qk_norm_rope(k_out=X, q_out=X, k=X, q=X)):
        with pytest.raises(ValueError, match="q: not on the GPU"):
            call()


def test_what_is_no_tensor_or_no_handle(lc, handle):
    for bad in (None, 3, "x", object()):
        with pytest.raises(ValueError, match="q: needs a tensor"):
            lc.ar_qk_norm_rope(bad, X, X, X)
        with pytest.raises(ValueError, match="h: needs a handle"):
            lc.ar_kv4_append(bad, X, X, I, X, X)
    with pytest.raises(ValueError, match="needs a tensor"):
        lc.ar_page_tables(*[None] * 11, 16)


def test_types_and_shapes(lc, handle):
    for bad in (X.half(), X.double(), X.int()):
        with pytest.raises(ValueError, match="dtype"):
            lc.ar_qk_norm_rope(bad, X, X, X)
    for bad in (X[0], X[None], torch.zeros(())):
        with pytest.raises(ValueError, match="q: needs"):
            lc.ar_qk_norm_rope(bad, X, X, X)
    with pytest.raises(ValueError, match="head_dim 128, got 64"):
        lc.ar_kv4_attention(handle, X[..., :64], X, X, I, I, I, X)
    with pytest.raises(ValueError, match="table"):
        lc.ar_kv4_attention(handle, X, X, X, I, I, I, X)


def test_a_destroyed_handle_is_refused(lc):
    h = lc.ar_kv4_create(2, 128, 16)
    lc.ar_kv4_destroy(h)
    lc.ar_kv4_destroy(h)  # as destroying nothing
    with pytest.raises((ValueError, lc.ArError)):
        lc.ar_kv4_append(h, X, X, I, X, X)


def test_signatures_are_documented(lc):
    for name in lc.DECODE_EXPORTS:
        fn = getattr(lc, name)
        assert fn.__name__ == name
    assert "scale=None" in lc.ar_kv4_attention.__text_signature__
