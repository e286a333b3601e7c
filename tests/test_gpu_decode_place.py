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
