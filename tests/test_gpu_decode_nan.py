"""ar_kv4_attention's logarithms where scores are NaN: a row that sees a NaN has NaN for its sum, so
NaN for its logarithm, and minus infinity stays the mark of a row that sees nothing. Both kinds of
tiles, against the plain 64-bit form."""

import pytest
import torch

from tests.test_gpu_decode_attention import BF, F32, Case
from tests.test_gpu_decode_chunks import Chunks

pytestmark = pytest.mark.gpu

KINDS = [(Case, BF), (Case, F32), (Chunks, BF)]


@pytest.fixture(scope="module")
def lc():
    import latency_collectives_amd as lc

    return lc


def _nan_keys(c, request, positions):
    """Keys of `request` at these positions become NaN, their values one."""
    slots = [int(c.table[request, p // c.page]) * c.page + p % c.page for p in positions]
    n = len(slots)
    k = torch.full((n, c.hkv, c.d), float("nan"), device="cuda")
    c.lc.ar_kv4_append(c.h, k, torch.ones_like(k), torch.tensor(slots, device="cuda"), c.data, c.scales)


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("kv", [70, 5000])
def test_nan_queries(lc, kind, dtype, kv):
    """Every score of these rows is NaN, in one workgroup and in parts."""
    c = kind(lc, [(70, kv), (3, 5)], 8, 2, 128, 16, dtype)
    c.q[1, 0, 3], c.q[2, 5, 100], c.q[69, 7] = float("nan"), float("inf"), float("nan")
    c.q[71, 3, 0] = float("nan")
    c.call().check()
    for row in ((1, 0), (2, 5), (69, 7), (71, 3)):
        assert torch.isnan(c.lse[row]), row
    assert int(torch.isnan(c.lse).sum()) == 4
    c.done()


@pytest.mark.parametrize("kind,dtype", KINDS)
def test_rows_whose_only_visible_keys_are_nan(lc, kind, dtype):
    """The first rows of a prompt, and with a window rows in the middle of one; a row that sees
    nothing beside them."""
    c = kind(lc, [(90, 90), (75, 60)], 4, 2, 64, 16, dtype)
    _nan_keys(c, 0, [0])
    c.call().check()
    assert torch.isnan(c.lse[:90]).all()
    assert torch.isneginf(c.lse[90:105]).all() and torch.isfinite(c.lse[105:]).all()
    c.done()
    c = kind(lc, [(90, 90), (75, 60)], 4, 2, 64, 16, dtype)
    _nan_keys(c, 0, range(20, 50))
    c.call(window=4).check()
    assert torch.isnan(c.lse[20:53]).all()
    assert torch.isfinite(c.lse[:20]).all() and torch.isfinite(c.lse[53:90]).all()
    c.done()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_single_token_of_a_nan_key(lc, dtype):
    c = Case(lc, [(1, 1), (1, 1), (1, 0)], 4, 2, 128, 16, dtype)
    _nan_keys(c, 1, [0])
    c.call().check()
    assert torch.isfinite(c.lse[0]).all() and torch.isnan(c.lse[1]).all() and torch.isneginf(c.lse[2]).all()
    c.done()


@pytest.mark.parametrize("kind,dtype", KINDS)
@pytest.mark.parametrize("first,last", [(0, 4095), (4095, 20000), (0, 20000), (33, 34)])
def test_parts_of_a_row_that_see_only_nan(lc, kind, dtype, first, last):
    """One long request cut over many workgroups; the NaN keys fill some of the parts, all, or a
    place of one."""
    c = kind(lc, [(17, 20000), (1, 9)], 16, 1, 64, 64, dtype)
    _nan_keys(c, 0, range(first, last))
    c.call().check()
    assert torch.isnan(c.lse[:17] if last < 20000 else c.lse[1:17]).all()
    assert torch.isfinite(c.lse[17]).all()
    c.done()
