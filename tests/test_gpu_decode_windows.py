"""ar_kv4_attention with windows in tiles of 128 rows, and windows, lengths and tables at the ends of
their range with either kind of tiles, against the plain 64-bit form. `large_tiles` repeats the rule by which
the call picks its tiles, so that a case here says which it reaches."""

import os
import re

import pytest
import torch

from tests import decode_ref as R
from tests.test_gpu_decode_attention import BF, F32, Case

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lc():
    import latency_collectives_amd as lc

    return lc


def large_tiles(c, window):
    """Whether the call takes the tiles of 128 rows: choose() of ar_decode_attn.hip."""
    with open(os.path.join(ROOT, "latency_collectives_amd", "csrc_decode", "ar_decode_attn.hip")) as f:
        many_tiles, shift = re.search(r"kManyTiles = (\d+), kManyUnits = 1 << (\d+)", f.read()).groups()
    nreq, tokens = len(c.new), c.q.shape[0]
    each = -(-tokens * (c.q.shape[1] // c.hkv) // nreq)
    if c.q.dtype != BF or each <= 128:
        return False
    tiles = -(-each // 128) * min(nreq, tokens) * c.hkv
    room = c.table.shape[1] * c.page
    units = (min(room, window) if window > 0 else room) // 32 + 1
    return (tiles >= int(many_tiles) and units >= 16) or tiles * units >= 1 << int(shift)


class Wide(Case):
    """A case whose table has room for `room` tokens a request, its columns past a request's pages out
    of range."""

    def __init__(self, lc, reqs, hq, hkv, d, page, dtype, room, **kw):
        super().__init__(lc, reqs, hq, hkv, d, page, dtype, **kw)
        n, width = self.table.shape
        wide = torch.full((n, max(width, -(-room // page))), -1, dtype=torch.int32, device="cuda")
        wide[:, 3::5] = MOST
        wide[:, :width] = self.table
        self.table = wide

    def check_rows(self, rows):
        """These rows of the step's tokens alone: token i of m is what a single new token of a request
        of length kv - m + i + 1 is."""
        starts = self.q_start.tolist()
        who = [max(b for b in range(len(self.new)) if starts[b] <= r and self.new[b] > 0) for r in rows]
        lens = [self.kv[b] - self.new[b] + r - starts[b] + 1 for r, b in zip(rows, who)]
        k, v = R.unpack(self.data.cpu(), self.scales.cpu(), self.page)
        out, lse, bound, lse_bound = R.attention(self.q[rows].cpu(), k, v, self.table[who].cpu(), lens,
                                                 list(range(len(rows) + 1)), self.page, self.scale, self.window)
        got, got_lse = self.out[rows].cpu().double(), self.lse[rows].cpu().double()
        assert torch.equal(torch.isnan(got), torch.isnan(out))
        assert not ((got - out).abs() > bound).any()
        assert torch.equal(torch.isneginf(got_lse), torch.isneginf(lse))
        assert torch.equal(torch.isnan(got_lse), torch.isnan(lse))
        assert not ((got_lse - lse).abs() > lse_bound)[torch.isfinite(lse)].any()
        return self


@pytest.mark.parametrize("window", [MOST, MOST - 1, MOST - 30, 1 << 30])
def test_the_largest_windows_beside_rows_below_position_zero(lc, window):
    """As no window: rows before the first position see nothing, the others of their tile all."""
    for dtype in (BF, F32):
        c = Case(lc, [(40, 20), (3, -5), (2, 30), (17, 17)], 6, 2, 128, 16, dtype).call(window=window).check()
        assert (c.out[:20] == 0).all() and (c.out[20:40] != 0).any()
        c.done()
    c = Wide(lc, [(1100, 600), (1100, 1100)], 32, 8, 64, 16, BF, 8192).call(window=window)
    assert large_tiles(c, window)
    assert (c.out[:500] == 0).all()
    c.check_rows([0, 499, 500, 501, 530, 531, 532, 700, 1099, 1100, 1600, 2199]).done()


@pytest.mark.parametrize("kv", [MOST, MOST - 1, MOST - 1700, MOST - 5000, 1 << 24])
def test_windows_that_begin_past_the_table(lc, kv):
    """Lengths up to the type's end over a short table: what the windows hold counts as masked."""
    for dtype in (BF, F32):
        c = Case(lc, [(1, 40), (3, 77), (20, 90)], 6, 2, 64, 16, dtype)
        c.kv_len[0] = c.kv_len[2] = c.kv[0] = c.kv[2] = kv
        c.call(window=33).check()
        assert (c.out[0] == 0).all() and torch.isneginf(c.lse[4:]).all() and (c.out[1:4] != 0).any()
        c.done()
    c = Wide(lc, [(1100, 600), (1100, 1100)], 32, 8, 64, 16, BF, 8192)
    c.kv_len[0] = c.kv[0] = kv
    c.call(window=500)
    assert large_tiles(c, 500)
    assert (c.out[:1100] == 0).all() and torch.isneginf(c.lse[:1100]).all()
    c.check_rows([0, 1099, 1100, 1599, 1600, 1601, 1700, 2199]).done()


def test_lengths_past_the_table(lc):
    """The same without a window: a row sees what the table holds."""
    c = Case(lc, [(1, 40), (20, 90)], 6, 2, 64, 16, BF)
    c.kv_len[:] = MOST
    c.kv = [MOST] * 2
    c.call().check().done()
    c = Wide(lc, [(1100, 600), (1100, 1100)], 32, 8, 64, 16, BF, 8192)
    c.kv_len[0] = c.kv[0] = MOST
    c.call()
    assert large_tiles(c, 0)
    c.check_rows([0, 31, 32, 1099, 1100, 1600, 2199]).done()


@pytest.mark.parametrize("hq,hkv", [(2, 1), (16, 8), (48, 24)])
@pytest.mark.parametrize("window", [0, 700])
def test_tables_so_wide_that_units_grow(lc, hq, hkv, window):
    """Tables for 2^31 tokens a request: with 33 jobs and more the sums of all requests' units of 32 tokens
    would pass 31 bits, so they are counted in units of 128 tokens (8 kv heads) or 512 (24)."""
    reqs = [(1, 5000), (3, 100), (1, 0), (9, 9), (40, 2100), (1, 127), (1, 129), (2, 4097)]
    for dtype in (BF, F32):
        c = Wide(lc, reqs, hq, hkv, 64, 1024, dtype, MOST).call(window=window)
        assert not large_tiles(c, window)
        c.check_rows([0, 1, 3, 4, 5, 12, 13, 14, 20, 53, 54, 55, 56, 57]).done()


@pytest.mark.parametrize("hq,hkv", [(16, 2), (24, 12)])
def test_wide_tables_with_large_tiles(lc, hq, hkv):
    reqs = [(140, 5000), (90, 100), (1, 0), (200, 200), (333, 2100), (1, 127), (64, 4097)]
    c = Wide(lc, reqs, hq, hkv, 64, 1024, BF, MOST).call()
    assert large_tiles(c, 0)
    c.check_rows([0, 1, 127, 139, 140, 150, 229, 230, 231, 240, 430, 431, 500, 763, 764, 765, 828]).done()


@pytest.mark.parametrize("window", [480, 481, 500, 639, 1000, 1100])
@pytest.mark.parametrize("kv", [1100, 1101, 1937])
def test_windows_in_large_tiles(lc, window, kv):
    """One prompt, from nothing and after a prefix: tiles whose windows begin inside a unit, rows of one
    wave with different windows, a length of work that grows and then stays."""
    c = Wide(lc, [(1100, kv)], 64, 8, 64, 16, BF, 2048, seed=window).call(window=window)
    assert large_tiles(c, window)
    c.check_rows([0, 1, 15, 16, 31, 32, 33, 470, 479, 480, 481, 500, 512, 600, 777, 1001, 1098, 1099]).done()


@pytest.mark.parametrize("d", [96, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 256])
def test_windows_in_large_tiles_of_other_heads(lc, d, page):
    c = Wide(lc, [(700, 900), (5, 5), (900, 900), (1, 800)], 40, 8, d, page, BF, 2048, seed=d).call(window=523)
    assert large_tiles(c, 523)
    c.check_rows([0, 7, 320, 323, 324, 699, 700, 704, 705, 706, 1000, 1227, 1228, 1229, 1300, 1604, 1605]).done()


@pytest.mark.parametrize("tokens,hq,hkv,window", [(4096, 32, 8, 4096), (8192, 32, 8, 1024), (3001, 32, 16, 777)])
def test_long_prompts_with_windows(lc, tokens, hq, hkv, window):
    """A window's work grows over the first tiles and stays for the others, which the split takes for a
    straight line: what it leaves out goes to a tile's last part. The same bits twice."""
    c = Wide(lc, [(tokens, tokens)], hq, hkv, 64, 16, BF, 0).call(window=window)
    assert large_tiles(c, window)
    first, first_lse = c.out.clone(), c.lse.clone()
    c.out.fill_(7.0), c.lse.fill_(7.0)
    c.call(window=window)
    assert torch.equal(c.out, first) and torch.equal(c.lse, first_lse)
    some = sorted({0, 1, 63, 64, 500, window - 1, window % tokens, (window + 1) % tokens, 2 * window % tokens,
                   tokens // 2, tokens - 33, tokens - 1})
    c.check_rows(some).done()


def test_windows_and_nan_in_large_tiles(lc):
    """NaN keys and values where some rows' windows hold them and others' have passed them."""
    for which in (0, 1):
        c = Wide(lc, [(1100, 1300)], 64, 8, 64, 16, BF, 2048)
        pos = [400, 901]
        slots = torch.tensor([int(c.table[0, p // 16]) * 16 + p % 16 for p in pos], device="cuda")
        kv = torch.ones(2, 2, 8, 64, device="cuda")
        kv[which, 0, :, 5], kv[which, 1, 3, 40] = float("nan"), float("nan")
        c.lc.ar_kv4_append(c.h, kv[0], kv[1], slots, c.data, c.scales)
        c.call(window=490)
        assert large_tiles(c, 490)
        # row r is at position r + 200; windows that hold 400 begin at rows 200, end at 689
        c.check_rows([0, 199, 200, 201, 300, 400, 688, 689, 690, 691, 700, 701, 702, 1000, 1099])
        assert torch.isnan(c.out[200:690, :, :32]).all() and not torch.isnan(c.out[:200]).any()
        if which == 1:
            assert not torch.isnan(c.out[:, :24, 32:]).any() and torch.isfinite(c.lse).all()
            assert torch.isnan(c.out[701:, 24:32, 32:]).all()
        c.done()


@pytest.mark.parametrize("window", [500, 900])
def test_rows_that_see_nothing_with_windows_in_large_tiles(lc, window):
    c = Wide(lc, [(700, 150), (600, 0), (300, -7), (500, 1200)], 64, 8, 64, 16, BF, 2048).call(window=window)
    assert large_tiles(c, window)
    assert (c.out[:550] == 0).all() and (c.out[700:1600] == 0).all()
    assert torch.isneginf(c.lse[:550]).all() and torch.isneginf(c.lse[700:1600]).all()
    c.check_rows([0, 549, 550, 551, 580, 699, 700, 1299, 1300, 1599, 1600, 1601, 1800, 2099]).done()
