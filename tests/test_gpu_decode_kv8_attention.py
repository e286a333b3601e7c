"""ar_kv8_attention on the GPU against the plain 64-bit form, within the bound that its roundings give
(decode_ref.attention: the same arithmetic as over the 4-bit cache). Whatever no request holds stands for NaN,
the places behind a request's last token in its own block among it."""

import math

import pytest
import torch

from tests import decode_ref as R
from tests import serving_ref as S
from tests.test_gpu_decode_attention import LENGTHS
from tests.test_gpu_decode_attention import Case as Case4

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lc():
    import latency_collectives_amd as lc

    return lc


class Case(Case4):
    """Requests (new tokens, length) over an 8-bit cache, pages in random order."""

    def __init__(self, lc, reqs, hq, hkv, d, page, dtype, seed=0, spare=3, sharp=1.0, room=0, vary=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lc, self.page, self.hkv, self.d = lc, page, hkv, d
        self.h = lc.ar_kv8_create(hkv, d, page)
        self.new, self.kv = [r[0] for r in reqs], [r[1] for r in reqs]
        held = [-(-max(n, 0) // page) for n in self.kv]
        pages = sum(held) + spare
        ids = torch.randperm(pages, generator=g).tolist()
        width = max(max(held), 1, -(-room // page))
        table, slots, tails, at = [], [], [], 0
        for n, p in zip(self.kv, held):
            mine = ids[at:at + p]
            at += p
            table.append(mine + [2 ** 31 - 1, -1, pages][at % 3:at % 3 + 1] * (width - p))
            slots += [mine[t // page] * page + t % page for t in range(max(n, 0))]
            tails += [mine[t // page] * page + t % page for t in range(max(n, 0), p * page)]
        self.data, self.scales = lc.ar_kv8_cache(self.h, pages)
        self.data.fill_(0x7F), self.scales.fill_(0xFF)  # NaN, and a scale that nothing writes
        n = len(slots)
        if n:
            k, v = (torch.randn(n, hkv, d, generator=g) for _ in range(2))
            size = torch.exp(vary * torch.randn(n, hkv, 1, generator=g))
            v = (v * size + torch.linspace(-1, 1, d)).cuda()
            lc.ar_kv8_append(self.h, k.cuda(), v, torch.tensor(slots, device="cuda"), self.data, self.scales)
        if tails:
            t = torch.tensor(tails, device="cuda")
            pg, off = t // page, t % page
            self.data[:, :, 0].view(pages, hkv, page, d)[pg, :, off] = 0xFF
            self.data[:, :, 1].view(pages, hkv, page // 4, d, 4)[pg, :, off // 4, :, off % 4] = 0x7F
        t = sum(self.new)
        self.q = (sharp * torch.randn(t, hq, d, generator=g)).to(dtype).cuda()
        self.table = torch.tensor(table, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(self.kv, dtype=torch.int32, device="cuda")
        starts = [0]
        for m in self.new:
            starts.append(starts[-1] + m)
        self.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.out = torch.full_like(self.q, 7.0)
        self.lse = torch.full((t, hq), 7.0, device="cuda")

    def call(self, scale=None, window=0, q=None, out=None, lse=None):
        self.scale = 1 / math.sqrt(self.d) if scale is None else scale
        self.window = window
        self.lc.ar_kv8_attention(self.h, self.q if q is None else q, self.data, self.scales, self.table,
                                 self.kv_len, self.q_start, self.out if out is None else out,
                                 self.lse if lse is None else lse, scale, window)
        return self

    def want(self):
        x, _ = S.unpack(self.data.cpu(), self.scales.cpu(), self.d)
        return R.attention(self.q.cpu(), x[:, :, 0], x[:, :, 1], self.table.cpu(), self.kv, self.q_start.tolist(),
                           self.page, self.scale, self.window)

    def poke(self, request, token, head, which, element):
        """A NaN code in a request's key or value."""
        pg, off = int(self.table[request, token // self.page]), token % self.page
        if which == 0:
            self.data[pg, head, 0].view(self.page, self.d)[off, element] = 0x7F
        else:
            self.data[pg, head, 1].view(self.page // 4, self.d, 4)[off // 4, element, off % 4] = 0xFF

    def done(self):
        torch.cuda.synchronize()
        self.lc.ar_kv8_destroy(self.h)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("hq,hkv,page", [(1, 1, 16), (8, 1, 64), (6, 2, 16), (34, 2, 32), (71, 1, 1024)])
def test_single_tokens(lc, dtype, d, hq, hkv, page):
    Case(lc, LENGTHS, hq, hkv, d, page, dtype, seed=d + hq).call().check().done()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("hq,hkv,page,window", [(4, 2, 16, 0), (5, 1, 32, 0), (3, 3, 16, 1), (16, 2, 64, 33),
                                                (8, 1, 16, 100)])
def test_several_tokens(lc, dtype, d, hq, hkv, page, window):
    reqs = [(3, 3), (0, 40), (7, 50), (40, 40), (1, 1), (33, 200), (70, 90), (2, 64), (0, 0)]
    Case(lc, reqs, hq, hkv, d, page, dtype, seed=d + window).call(window=window).check().done()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [0, 5])
def test_rows_that_see_nothing(lc, dtype, window):
    """More new tokens than the length, lengths of zero and below, no requests' tokens at all."""
    reqs = [(4, 2), (1, 0), (3, -5), (40, 20), (2, 30), (17, 17)]
    c = Case(lc, reqs, 6, 2, 128, 16, dtype).call(window=window).check()
    assert (c.out[:2] == 0).all() and (c.out[4] == 0).all() and (c.out[2] != 0).any()
    c.done()
    Case(lc, [(0, 0), (0, 5)], 2, 1, 64, 16, dtype).call().check().done()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kv,window", [(5000, 0), (20000, 0), (20000, 4099)])
def test_long_sequences_in_parts(lc, dtype, kv, window):
    """One request's tokens cut over many workgroups, beside short ones; a second call finds the
    workspace as the first did and gives the same bits."""
    c = Case(lc, [(1, kv), (1, 3), (5, 700), (1, 0)], 8, 1, 128, 64, dtype).call(window=window).check()
    first, first_lse = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.out.fill_(7.0), c.lse.fill_(7.0)
        c.call(window=window)
        assert torch.equal(c.out, first) and torch.equal(c.lse, first_lse)
    c.done()


@pytest.mark.parametrize("scale,sharp", [(1.0, 3.0), (0.0, 1.0), (-0.5, 1.0), (30.0, 2.0)])
def test_scales_and_sharp_rows(lc, scale, sharp):
    for dtype in (BF, F32):
        Case(lc, [(1, 900), (9, 333)], 4, 2, 64, 16, dtype, sharp=sharp).call(scale=scale).check().done()


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("hkv,group,reqs,window", [
    (2, 4, [(300, 700), (129, 129), (33, 2000), (256, 260)], 0),
    (2, 4, [(300, 700), (129, 129), (33, 2000), (256, 260)], 77),
    (1, 3, [(1000, 1000), (1, 1), (517, 40), (0, 9)], 0),  # rows before position 0 see nothing
])
def test_tiles_of_128_rows(lc, d, hkv, group, reqs, window):
    """Prompt chunks; the table's room makes the call take the tiles of 128 rows."""
    Case(lc, reqs, hkv * group, hkv, d, 32, BF, seed=d, room=1 << 19).call(window=window).check().done()


@pytest.mark.parametrize("scale", [-0.2, 0.0, 2.0])
def test_tiles_of_128_rows_at_other_scales(lc, scale):
    Case(lc, [(150, 400), (200, 200)], 4, 1, 128, 16, BF, room=1 << 19).call(scale=scale).check().done()


@pytest.mark.parametrize("room", [0, 1 << 19])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_nan_keys_and_values_reach_only_rows_that_see_them(lc, dtype, d, room):
    """A NaN element of a key makes NaN the rows that see it, one of a value its own element of them, and
    nothing else: not earlier tokens of the same tile, not rows whose window has passed it, not others."""
    for which, window in ((0, 0), (1, 0), (1, 8), (0, 8), (1, 40)):
        c = Case(lc, [(200, 230), (1, 60), (130, 130)], 2, 1, d, 16, dtype, room=room, seed=which)
        for token in (31, 100, 229):
            c.poke(0, token, 0, which, d - 3)
        c.poke(1, 59, 0, which, 5)
        c.poke(2, 64, 0, which, 0)
        c.call(window=window).check()
        assert torch.isnan(c.out).any() and not torch.isnan(c.out).all()
        c.done()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_page_ids_out_of_range_count_as_masked(lc, dtype):
    c = Case(lc, [(1, 300), (40, 200)], 4, 2, 128, 16, dtype)
    c.table[0, 3], c.table[0, 18], c.table[1, 0], c.table[1, 5] = -1, 2 ** 31 - 1, -2 ** 31, 999999
    c.call().check().done()


@pytest.mark.parametrize("vary", [0.0, 6.0])
def test_values_of_very_different_sizes(lc, vary):
    """Blocks whose scales lie far apart, in one tile."""
    for room in (0, 1 << 19):
        Case(lc, [(140, 500), (1, 333)], 2, 1, 128, 64, BF, vary=vary, room=room).call().check().done()


def test_strided_queries_and_outputs(lc):
    c = Case(lc, [(1, 77), (5, 50)], 6, 2, 128, 16, BF)
    wide = torch.zeros(6, 6, 400, dtype=BF, device="cuda")
    q, out = wide[..., 8:136], torch.full((6, 6, 256), 5.0, dtype=BF, device="cuda")
    q.copy_(c.q)
    c.call()
    c.lc.ar_kv8_attention(c.h, q, c.data, c.scales, c.table, c.kv_len, c.q_start, out[..., 64:192], c.lse)
    assert torch.equal(out[..., 64:192], c.out)
    assert (out[..., :64] == 5).all() and (out[..., 192:] == 5).all()
    c.done()


def test_tokens_without_a_request_keep_their_rows(lc):
    c = Case(lc, [(2, 30), (3, 40)], 4, 1, 64, 16, BF)
    c.q_start = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    c.call()
    torch.cuda.synchronize()
    assert (c.out[4] == 7).all() and (c.lse[4] == 7).all() and (c.out[:4] != 7).any()
    c.done()


@pytest.mark.parametrize("kind", [Case, Case4])
@pytest.mark.parametrize("room", [0, 1 << 19])
def test_starts_that_are_out_of_order_or_range(lc, kind, room):
    """Starts are taken between 0 and ntokens, an end before its start is a request without tokens."""
    for starts in ([-5, 200, 2 ** 31 - 1], [10, 60, 60], [250, -2 ** 31, 250], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1],
                   [7, -2 ** 31, -2 ** 31]):
        c = kind(lc, [(200, 300), (50, 90)], 4, 2, 64, 16, BF)
        if room:  # a wider table takes the call to the tiles of 128 rows
            wide = torch.full((2, room // 16), -1, dtype=torch.int32, device="cuda")
            wide[:, :c.table.shape[1]] = c.table
            c.table = wide
        c.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        c.call()
        torch.cuda.synchronize()
        at = [min(max(x, 0), 250) for x in starts]
        free = torch.ones(250, dtype=torch.bool, device="cuda")
        for a, b in zip(at, at[1:]):
            free[a:b] = False
        assert (c.out[free] == 7).all() and (c.out[~free] != 7).any(-1).all()
        c.done()


def test_captured_and_replayed(lc):
    """One captured call, replayed over new lengths and queries between other work on the same handle."""
    c = Case(lc, [(1, 3000), (1, 700)], 8, 1, 128, 16, BF)
    other = Case(lc, [(4, 900)], 8, 1, 128, 16, BF, seed=9)
    c.call()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.call()
    for i in range(4):
        c.kv = [3000 - 450 * i, 700 - i]
        c.kv_len.copy_(torch.tensor(c.kv, dtype=torch.int32))
        c.q.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = c.out.clone()
        lc.ar_kv8_attention(c.h, other.q, other.data, other.scales, other.table, other.kv_len, other.q_start, other.out)
        c.call()
        torch.cuda.synchronize()
        assert torch.equal(c.out, got), i
        c.check()
    other.done()
    c.done()


def test_a_large_cache(lc):
    """Pages beyond 2^31 bytes of data."""
    heads, d, page = 8, 128, 1024
    pages = (1 << 31) // (heads * 2 * page * d) + 40
    h = lc.ar_kv8_create(heads, d, page)
    data, scales = lc.ar_kv8_cache(h, pages)
    k, v = (torch.randn(64, heads, d, device="cuda") for _ in range(2))
    high, low = (torch.arange(64, device="cuda") + p * page for p in (pages - 1, 0))
    outs = []
    q = torch.randn(1, 16, d, device="cuda")
    for slots in (high, low):
        lc.ar_kv8_append(h, k, v, slots, data, scales)
        out = torch.empty_like(q)
        table = (slots[:1] // page).int()[:, None]
        lc.ar_kv8_attention(h, q, data, scales, table, torch.tensor([64], dtype=torch.int32, device="cuda"),
                            torch.tensor([0, 1], dtype=torch.int32, device="cuda"), out)
        outs.append(out)
    assert torch.equal(data[0], data[-1]) and torch.equal(outs[0], outs[1])
    kk, vv = torch.empty_like(k), torch.empty_like(v)
    lc.ar_kv8_read(h, high, data, scales, kk, vv)
    assert ((kk - k).abs() <= 2.0 ** -4 * k.abs() + 2.0 ** -8).all()
    torch.cuda.synchronize()
    lc.ar_kv8_destroy(h)
