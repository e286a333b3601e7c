"""The decode operators and the GPU that a call's tensors, its handle and its stream belong to."""

import pytest
import torch

from tests.test_gpu_decode_attention import BF, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lc():
    import latency_collectives_amd as lc

    return lc


def test_a_handle_of_another_gpu_is_refused(lc):
    """Its workspace is on its own GPU. The handle says here that it was made on the next one."""
    c = Case(lc, [(1, 40), (3, 50)], 4, 2, 64, 16, BF).call().check()
    assert c.h.device == torch.cuda.current_device()
    want = c.out.clone()
    c.h.device += 1
    c.out.fill_(7.0)
    with pytest.raises(ValueError, match="h: made on GPU 1, the tensors are on GPU 0"):
        c.call()
    assert (c.out == 7.0).all()
    c.h.device -= 1
    c.call()
    assert torch.equal(c.out, want)
    c.done()


@pytest.mark.skipif("torch.cuda.device_count() < 2", reason="needs two GPUs")
def test_calls_go_to_the_gpu_of_their_tensors(lc):
    from latency_collectives_amd import _decode
    from tests.test_decode_host import _attn

    with torch.cuda.device(1):
        c = Case(lc, [(1, 40), (3, 50)], 4, 2, 64, 16, BF).call().check()
        want = c.out.clone()
        c.out.fill_(7.0)
    c.call()  # with GPU 0 current
    assert torch.equal(c.out, want) and torch.cuda.current_device() == 0
    rc = _decode._entry.ar_kv4_attention(c.h, _decode._ATTENTION.pack(*_attn(hq=4)), None)
    assert rc == lc.AR_EINVAL and "GPU 1" in lc.ar_last_error()
    c.done()


def test_strides_of_one_token_or_one_head_do_not_count(lc):
    """torch lets a dimension of size one have any stride; a slice of a wider buffer keeps its pitch."""
    d, n = 64, 6 * 64
    wide = torch.randn(5, n + 3, device="cuda").to(BF)
    q, k, v = (wide.as_strided((1, h, d), (n + 3, d, 1), at * d) for h, at in ((4, 0), (1, 4), (1, 5)))
    assert q.stride(0) % 4 == 3
    plain = [x.contiguous() for x in (q, k, v)]
    outs = []
    for a, b, c in ((q, k, v), plain):
        qo, ko = torch.zeros(1, 4, d, dtype=BF, device="cuda"), torch.zeros(1, 1, d, dtype=BF, device="cuda")
        lc.ar_qk_norm_rope(a, b, qo, ko, q_weight=torch.ones(d, dtype=BF, device="cuda"))
        h = lc.ar_kv4_create(1, d, 16)
        data, scales = lc.ar_kv4_cache(h, 2)
        lc.ar_kv4_append(h, b, c, torch.tensor([5], device="cuda"), data, scales)
        # one head a kv head: its stride is not used either
        one = a.as_strided((1, 1, d), (n + 3, 7, 1))
        out = torch.zeros(1, 1, d, dtype=BF, device="cuda").as_strided((1, 1, d), (13, 5, 1))
        table, kv, starts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[0]], [6], [0, 1]))
        lc.ar_kv4_attention(h, one, data, scales, table, kv, starts, out)
        outs.append([qo, ko, data, scales, out])
        torch.cuda.synchronize()
        lc.ar_kv4_destroy(h)
    for x, y in zip(*outs):
        assert torch.equal(x, y)
