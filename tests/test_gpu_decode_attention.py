"""ar_kv4_attention on the GPU against the plain 64-bit form, within the bound that its roundings
give (decode_ref.attention). Caches are filled with bytes that stand for NaN and tables with page
ids out of range wherever a request holds nothing."""

import math

import pytest
import torch

from tests import decode_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lc():
    import latency_collectives_amd as lc

    return lc


class Case:
    """Requests (new tokens, length) over a cache of quantised values, pages in random order."""

    def __init__(self, lc, reqs, hq, hkv, d, page, dtype, seed=0, spare=3, sharp=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lc, self.page, self.hkv, self.d = lc, page, hkv, d
        self.h = lc.ar_kv4_create(hkv, d, page)
        self.new, self.kv = [r[0] for r in reqs], [r[1] for r in reqs]
        held = [-(-max(n, 0) // page) for n in self.kv]
        pages = sum(held) + spare
        ids = torch.randperm(pages, generator=g).tolist()
        width = max(max(held), 1)
        table, slots, at = [], [], 0
        for n, p in zip(self.kv, held):
            mine = ids[at:at + p]
            at += p
            table.append(mine + [2 ** 31 - 1, -1, pages][at % 3:at % 3 + 1] * (width - p))
            slots += [mine[t // page] * page + t % page for t in range(max(n, 0))]
        self.data, self.scales = lc.ar_kv4_cache(self.h, pages)
        self.data.fill_(0x77), self.scales.fill_(0xFE)  # what nothing wrote stands for NaN
        n = len(slots)
        if n:
            k, v = (torch.randn(n, hkv, d, generator=g).cuda() for _ in range(2))
            v += torch.linspace(-1, 1, d, device="cuda")
            lc.ar_kv4_append(self.h, k, v, torch.tensor(slots, device="cuda"), self.data, self.scales)
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
        self.lc.ar_kv4_attention(self.h, self.q if q is None else q, self.data, self.scales, self.table,
                                 self.kv_len, self.q_start, self.out if out is None else out,
                                 self.lse if lse is None else lse, scale, window)
        return self

    def want(self):
        k, v = R.unpack(self.data.cpu(), self.scales.cpu(), self.page)
        return R.attention(self.q.cpu(), k, v, self.table.cpu(), self.kv, self.q_start.tolist(), self.page,
                           self.scale, self.window)

    def check(self):
        out, lse, bound, lse_bound = self.want()
        got, got_lse = self.out.cpu().double(), self.lse.cpu().double()
        wrong = torch.isnan(got) != torch.isnan(out)
        assert not wrong.any(), f"NaN in other places: {int(wrong.sum())}"
        fine = ~torch.isnan(out)
        over = ((got - out).abs() - bound)[fine]
        assert over.numel() == 0 or float(over.max()) <= 0, float(over.max())
        dead = torch.isinf(lse)
        assert torch.equal(torch.isinf(got_lse) & (got_lse < 0), dead)
        live = ~dead & ~torch.isnan(lse)
        assert torch.equal(torch.isnan(got_lse), torch.isnan(lse))
        over = ((got_lse - lse).abs() - lse_bound)[live]
        assert over.numel() == 0 or float(over.max()) <= 0, float(over.max())
        return self

    def done(self):
        torch.cuda.synchronize()
        self.lc.ar_kv4_destroy(self.h)


LENGTHS = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 31), (1, 32), (1, 33), (1, 127), (1, 128),
           (1, 129), (1, 300)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("hq,hkv,page", [(1, 1, 16), (8, 1, 64), (6, 2, 16), (34, 2, 32), (71, 1, 1024)])
def test_single_tokens(lc, dtype, d, hq, hkv, page):
    Case(lc, LENGTHS, hq, hkv, d, page, dtype, seed=d + hq).call().check().done()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
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
    """Rows with one weight near 1, all weights equal, negative scales; the running maximum moves."""
    for dtype in (BF, F32):
        Case(lc, [(1, 900), (9, 333)], 4, 2, 64, 16, dtype, sharp=sharp).call(scale=scale).check().done()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nan_keys_and_values_reach_only_rows_that_see_them(lc, dtype):
    """A NaN key or value makes NaN what sees it (a value its 32 elements) and nothing else: not
    earlier tokens of the same tile, not rows whose window has passed it, not other requests."""
    for which, window in ((0, 0), (1, 0), (1, 8), (0, 8)):
        c = Case(lc, [(60, 100), (1, 40), (12, 12)], 4, 2, 128, 16, dtype)
        slot = int(c.table[0, 70 // 16]) * 16 + 70 % 16
        k, v = torch.ones(2, 1, 2, 128, device="cuda")
        (k, v)[which][0, 1, 40] = float("nan")
        c.lc.ar_kv4_append(c.h, k, v, torch.tensor([slot], device="cuda"), c.data, c.scales)
        c.call(window=window).check()
        assert torch.isnan(c.out).any() and not torch.isnan(c.out[:, :2]).any()
        assert not torch.isnan(c.out[:30]).any()
        c.done()


def test_extreme_queries_stay_in_their_rows(lc):
    """An infinite or NaN query, and products beyond binary32, spoil only their own row."""
    for dtype in (BF, F32):
        c = Case(lc, [(5, 200)], 4, 2, 64, 16, dtype)
        clean = c.call().out.clone()
        c.q[1, 0, 3], c.q[2, 1, 0], c.q[3, 3] = float("inf"), float("nan"), 3e38
        c.call()
        same = torch.ones(5, 4, dtype=torch.bool, device="cuda")
        same[1, 0] = same[2, 1] = same[3, 3] = False
        assert torch.equal(c.out[same], clean[same])
        assert torch.isnan(c.out[1, 0]).all() and torch.isnan(c.out[2, 1]).all()
        c.done()


def test_bad_pages_count_as_masked(lc):
    """Page ids out of range in the middle of a request, and lengths beyond the table."""
    for dtype in (BF, F32):
        c = Case(lc, [(2, 100), (1, 64), (3, 90)], 4, 1, 128, 16, dtype)
        c.table[0, 2], c.table[1, 0], c.table[1, 3] = -1, 1 << 30, c.data.shape[0]
        c.kv_len[2] = c.kv[2] = 3000
        c.call().check().done()
    c = Case(lc, [(1, 16)], 2, 1, 64, 16, BF)
    c.table.fill_(-3)
    c.call().check()
    assert (c.out == 0).all()
    c.done()


def test_strided_queries_and_outputs_and_no_lse(lc):
    for dtype in (BF, F32):
        c = Case(lc, [(3, 77), (1, 500), (20, 20)], 6, 2, 64, 32, dtype).call().check()
        t = c.q.shape[0]
        wide = torch.zeros(t, 10, 64, dtype=dtype, device="cuda")
        wide[:, 2:8] = c.q
        by_head = torch.full((6, t + 1, 64), 7.0, dtype=dtype, device="cuda")
        out = by_head[:, :t].transpose(0, 1)
        lc.ar_kv4_attention(c.h, wide[:, 2:8], c.data, c.scales, c.table, c.kv_len, c.q_start, out)
        assert torch.equal(out, c.out) and (by_head[:, t] == 7.0).all()
        c.done()


def test_tokens_that_no_request_covers_keep_their_rows(lc):
    c = Case(lc, [(2, 30), (3, 40)], 4, 2, 64, 16, BF).call().check()
    q = torch.cat([c.q, c.q])
    out = torch.full_like(q, 7.0)
    lse = torch.full((10, 4), 7.0, device="cuda")
    lc.ar_kv4_attention(c.h, q, c.data, c.scales, c.table, c.kv_len, c.q_start, out, lse)
    assert torch.equal(out[:5], c.out) and (out[5:] == 7.0).all() and (lse[5:] == 7.0).all()
    # starts out of range are bounded: nothing outside the tensors is touched
    bad = torch.tensor([3, -7, 99], dtype=torch.int32, device="cuda")
    lc.ar_kv4_attention(c.h, c.q, c.data, c.scales, c.table, c.kv_len, bad, c.out, c.lse)
    torch.cuda.synchronize()
    c.done()


def test_many_requests(lc):
    """More requests than a wave has lanes, ragged, some without tokens."""
    g = torch.Generator().manual_seed(1)
    reqs = [(int(m), int(n)) for m, n in zip(torch.randint(0, 3, (333,), generator=g),
                                             torch.randint(0, 70, (333,), generator=g))]
    Case(lc, reqs, 4, 2, 64, 16, BF).call().check().done()


def test_pages_beyond_32_bit_offsets(lc):
    heads, d, page = 8, 128, 64
    pages = (5 << 30) // (heads * page * d)
    c = Case(lc, [(1, 200), (4, 70)], 16, heads, d, page, BF)
    want, lse = c.call().check().out.clone(), c.lse.clone()
    n = c.data.shape[0]
    data = torch.empty(pages, *c.data.shape[1:], dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, *c.scales.shape[1:], dtype=torch.uint8, device="cuda")
    data[-n:], scales[-n:] = c.data, c.scales
    held = (c.table >= 0) & (c.table < n)
    c.table[held] += pages - n
    c.data, c.scales = data, scales
    c.out.fill_(7.0)
    c.call()
    assert torch.equal(c.out, want) and torch.equal(c.lse, lse)
    c.done()


def test_another_stream_and_graph_replays(lc):
    """On a stream of its own, and captured: replays with eager calls between them on the same
    handle, each for the lengths that its buffers hold then."""
    c = Case(lc, [(1, 3000), (1, 50), (2, 77)], 8, 1, 128, 16, BF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.call()
    side.synchronize()
    c.check()
    graph = torch.cuda.CUDAGraph()
    out, lse = torch.zeros_like(c.out), torch.zeros_like(c.lse)
    with torch.cuda.graph(graph):
        c.call(out=out, lse=lse)
    for lens in ([3000, 50, 77], [1, 17, 2], [2048, 0, 64], [3000, 50, 77]):
        c.kv_len.copy_(torch.tensor(lens)), c.q.copy_(torch.randn(c.q.shape))
        c.kv = lens
        graph.replay()
        torch.cuda.synchronize()
        c.call().check()
        assert torch.equal(out, c.out) and torch.equal(lse, c.lse)
    c.done()
