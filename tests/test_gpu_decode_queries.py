"""bfloat16 queries enter the attention's products as they are, whatever tiles a call takes: elements
far below the largest of their row count in full. Against the plain 64-bit form within the bound of
binary32 sums (decode_ref.attention), which the logarithms show best."""

import pytest
import torch

from tests.test_gpu_decode_attention import BF, Case
from tests.test_gpu_decode_windows import Wide, large_tiles

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lc():
    import latency_collectives_amd as lc

    return lc


def _both(lc, d, queries):
    """The same requests with either kind of tiles."""
    for wide in (False, True):
        reqs = [(70, 90), (64, 700)]
        c = Wide(lc, reqs, 8, 2, d, 16, BF, 1 << 21, seed=d) if wide else Case(lc, reqs, 8, 2, d, 16, BF, seed=d)
        c.q = queries(c.q.shape).to(BF).cuda()
        c.call()
        assert large_tiles(c, 0) == wide
        c.check().done()


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("factor", [100.0, 400.0, 2.0 ** 16])
def test_elements_beside_a_far_larger_one(lc, d, factor):
    g = torch.Generator().manual_seed(d)

    def queries(shape):
        q = torch.randn(shape, generator=g)
        q[..., 5::32] *= factor / 30
        q[..., 7] *= factor
        return q

    _both(lc, d, queries)


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
def test_elements_of_every_size(lc, d):
    """2^-30 to 2^4 of each other in one row, zero rows, rows of the smallest normal values."""
    g = torch.Generator().manual_seed(d)

    def queries(shape):
        q = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-30, 5, shape, generator=g).float())
        q[3] = 0.0
        q[5] = torch.randn(shape[1:], generator=g) * 2.0 ** -120
        return q

    _both(lc, d, queries)
