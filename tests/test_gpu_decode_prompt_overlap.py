"""ar_prompt_attention with requests that overlap: the rows of those that do not overlap are right all the same.
Starts that go back and forth (a, b, a, b, ..) are that many requests a .. b, and more tiles than the tokens have
otherwise."""

import pytest
import torch

from tests import serving_ref as S
from tests.test_gpu_decode_prompt_attention import Case, lc  # noqa: F401  (lc is the fixture)

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def alone(c, spans):
    """The rows of requests (a, b) that overlap nobody, against the 64-bit form of each request for itself."""
    for a, b in spans:
        out, lse, bound, lse_bound = S.prompt_attention(c.q[a:b].cpu(), c.k[a:b].cpu(), c.v[a:b].cpu(), [0, b - a],
                                                        c.scale, c.window)
        assert ((c.out[a:b].cpu().double() - out).abs() <= bound).all(), (a, b)
        assert ((c.lse[a:b].cpu().double() - lse).abs() <= lse_bound).all(), (a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("hq,hkv,times", [(8, 1, 3), (4, 2, 4), (8, 1, 40)])
def test_few_rows(lc, dtype, d, hq, hkv, times):  # noqa: F811
    """Requests before, between and behind those that overlap."""
    c = Case(lc, [120], hq, hkv, d, dtype)
    c.q_start = torch.tensor([0, 10] + [100, 10] * times + [100, 109, 113], dtype=torch.int32, device="cuda")
    c.call()
    alone(c, [(0, 10), (100, 109), (109, 113)])
    assert (c.out[113:] == 7).all() and (c.lse[113:] == 7).all()
    assert (c.out[10:100] != 7).any(-1).all() and (c.lse[10:100] != 7).all()  # by one of them at least
    c.call(window=5)
    alone(c, [(0, 10), (100, 109), (109, 113)])
    c.done()


@pytest.mark.parametrize("dtype,n", [(BF, 1600), (BF, 6000), (F32, 1600)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_rows(lc, dtype, n, d):  # noqa: F811
    """More rows than few; 6000 tokens of 64 heads take the large tiles."""
    c = Case(lc, [n], 64, 2, d, dtype)
    c.q_start = torch.tensor([0, 130] + [n - 200, 130] * 2 + [n - 200, n - 100, n - 99], dtype=torch.int32, device="cuda")
    c.call()
    alone(c, [(0, 130), (n - 200, n - 100), (n - 100, n - 99)])
    assert (c.out[n - 99:] == 7).all() and (c.out[130:n - 200] != 7).any(-1).all()
    c.done()


def test_more_requests_than_tokens(lc):  # noqa: F811
    """A thousand requests over a hundred tokens, a lane's requests several."""
    c = Case(lc, [100], 8, 1, 64, BF)
    c.q_start = torch.tensor([0, 10] + [90, 10] * 500 + [90, 100], dtype=torch.int32, device="cuda")
    c.call()
    alone(c, [(0, 10), (90, 100)])
    assert (c.out[10:90] != 7).any(-1).all()
    c.done()


def test_overlaps_without_end(lc):  # noqa: F811
    """Four thousand times the tokens: the call ends soon, with the rows of nobody's tokens as they were."""
    c = Case(lc, [100], 8, 1, 64, BF)
    c.q_start = torch.tensor([90, 0] * 5000, dtype=torch.int32, device="cuda")
    c.call()
    torch.cuda.synchronize()
    assert (c.out[90:] == 7).all() and (c.lse[90:] == 7).all()
    c.done()
