"""The life of a cache's pages on the GPU against plain lists (serving_ref): forks, frees and compactions give
equal numbers, copies equal bytes."""

import random

import pytest
import torch

from tests import serving_ref as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lc():
    import latency_collectives_amd as lc

    return lc


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class State:
    """A pool of pages on the GPU beside lists."""

    def __init__(self, lc, nreq, width, pages, page, stride=None):
        self.lc, self.nreq, self.width, self.pages, self.page = lc, nreq, width, pages, page
        order = list(range(pages))
        random.Random(pages).shuffle(order)
        self.free, self.pool, self.kv = order, [0, pages], [0] * nreq
        self.shares, self.table = [0] * pages, [[-1] * width for _ in range(nreq)]
        self.gfree, self.gpool, self.gkv, self.gshares = i32(order), i32(self.pool), i32(self.kv), i32(self.shares)
        whole = torch.full((nreq, stride or width), -1, dtype=torch.int32, device="cuda")
        self.gtable = whole[:, :width]
        self.scratch = lc.ar_pages_scratch(pages)

    def grow(self, new):
        """ar_page_tables, against the lists' own rule."""
        n = sum(new)
        out = [torch.full((m,), -7, dtype=t, device="cuda") for m, t in (
            (self.nreq, torch.int32), (self.nreq + 1, torch.int32), (n, torch.int64), (n, torch.int32),
            (2, torch.int32), (self.nreq, torch.int32))]
        self.lc.ar_page_tables(self.gkv, i32(new), self.gpool, self.gfree, self.gtable, *out, self.page)
        self.gkv, self.gpool = out[0], out[4]
        at = self.pool[0]
        for b, m in enumerate(new):
            for j in range(S.pages_for(self.kv[b], self.page), S.pages_for(self.kv[b] + m, self.page)):
                self.table[b][j] = self.free[at]
                at += 1
            self.kv[b] += m
        self.pool = [at, self.pool[1]]
        self.check()

    def fork(self, src, dst):
        kv, pool = torch.empty_like(self.gkv), torch.empty_like(self.gpool)
        lists = [torch.full((len(src),), -7, dtype=torch.int32, device="cuda") for _ in range(3)]
        self.lc.ar_pages_fork(i32(src), i32(dst), self.gkv, self.gtable, self.gshares, self.gpool, self.gfree, kv, pool,
                              *lists, self.page)
        self.gkv, self.gpool = kv, pool
        self.table, self.shares, self.kv, self.pool, *want = S.fork(src, dst, self.kv, self.table, self.shares,
                                                                    self.pool, self.free, self.page)
        assert [x.tolist() for x in lists] == want
        self.check()
        return lists

    def release(self, requests):
        kv, pool = torch.empty_like(self.gkv), torch.empty_like(self.gpool)
        self.lc.ar_pages_free(i32(requests), self.gkv, self.gtable, self.gshares, self.gpool, self.gfree, kv, pool,
                              self.scratch, self.page)
        self.gkv, self.gpool = kv, pool
        self.shares, self.free, self.kv, self.pool = S.free_pages(requests, self.kv, self.table, self.shares, self.pool,
                                                                  self.free, self.page)
        self.check()

    def compact(self):
        table, shares = torch.full_like(self.gtable, -7), torch.full_like(self.gshares, -7)
        moves = [torch.full((self.pages // 2 + 1,), -7, dtype=torch.int32, device="cuda") for _ in range(2)]
        pool = torch.empty_like(self.gpool)
        self.lc.ar_pages_compact(self.gkv, self.gtable, self.gshares, table, shares, self.gfree, pool, *moves,
                                 self.scratch, self.page)
        self.gtable, self.gshares, self.gpool = table, shares, pool
        self.table, self.shares, self.pool, *want = S.compact(self.kv, self.table, self.shares, self.page,
                                                              self.pages // 2 + 1)
        self.free = list(range(self.pages))
        assert [x.tolist() for x in moves] == want
        self.check()
        return moves

    def check(self):
        torch.cuda.synchronize()
        assert self.gkv.tolist() == self.kv
        assert self.gpool.tolist() == self.pool
        assert self.gtable.tolist() == self.table
        assert self.gshares.tolist() == self.shares
        assert self.gfree.tolist() == self.free
        assert not self.scratch.any()


@pytest.mark.parametrize("nreq,width,pages,page,stride", [(8, 9, 60, 16, None), (40, 20, 900, 4, 33), (5, 3, 31, 1, 3),
                                                          (3, 2, 32, 7, None)])
def test_lives_of_requests(lc, nreq, width, pages, page, stride):
    """Random steps: growth, forks (of empty requests, into taken rows, twice the same, out of range), frees, compactions."""
    rng = random.Random(nreq)
    s = State(lc, nreq, width, pages, page, stride)
    for step in range(14):
        room = s.pool[1] - s.pool[0]
        new = []
        for b in range(nreq):
            n = rng.choice([0, 0, 1, 2, page, rng.randrange(1, page * width + 1)])
            n = min(n, width * page - s.kv[b])
            need = S.pages_for(s.kv[b] + n, page) - S.pages_for(s.kv[b], page)
            # a shared last page is not written to: forks gave it a copy, so growth is always allowed
            if need > room:
                n = 0
                need = 0
            room -= need
            new.append(n)
        s.grow(new)
        k = rng.randrange(0, nreq + 3)
        s.fork([rng.randrange(-1, nreq + 1) for _ in range(k)], [rng.randrange(-1, nreq + 1) for _ in range(k)])
        if step % 3 != 0:
            s.release([rng.randrange(-1, nreq + 1) for _ in range(rng.randrange(0, nreq))])
        if step % 5 == 4:
            s.compact()
    s.release(list(range(nreq)))
    assert s.pool == [0, pages] and not any(s.shares)


def test_no_page_left_for_the_last_one(lc):
    s = State(lc, 6, 4, 7, 16)
    s.grow([20, 33, 0, 0, 0, 0])  # five pages
    _, _, refused = s.fork([0, 1, 0, 0], [2, 3, 4, 5])
    assert refused.tolist() == [0, 0, 1, 1]
    s.release([0, 1])
    s.release([2, 3])
    assert s.pool == [0, 7]


def test_whole_pages_need_none(lc):
    s = State(lc, 5, 4, 4, 16)
    s.grow([32, 17, 0, 0, 0])
    src, dst, refused = s.fork([1, 0, 0], [2, 3, 4])
    assert refused.tolist() == [1, 0, 0] and src.tolist() == [-1] * 3


@pytest.mark.parametrize("nreq", [1, 1000, 4096])
def test_many_requests(lc, nreq):
    s = State(lc, nreq, 3, 4 * nreq + 5, 16)
    half = nreq // 2
    s.grow([1 + b % 40 if b < max(half, 1) else 0 for b in range(nreq)])
    s.fork([b % max(half, 1) for b in range(half)], list(range(half, 2 * half)))
    s.release(list(range(0, nreq, 2)))
    s.compact()
    s.release(list(range(nreq)) * (1 if nreq > 2000 else 3))
    s.compact()


@pytest.mark.parametrize("pages", [1 << 19, (1 << 19) - 1, 70001])
def test_large_pools(lc, pages):
    """The largest pool, and ones that end inside a word."""
    nreq, width, page = 64, 1024, 16
    rng = random.Random(pages)
    table = torch.randperm(pages, device="cuda")[:nreq * width].view(nreq, width).int()
    kv = [rng.randrange(0, width * page + 1) for _ in range(nreq)]
    kv[0], kv[1] = width * page, 0
    shares = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table[5, :100] = table[0, :100]
    shares[table[0, :100].long()] = 1
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    scratch = lc.ar_pages_scratch(pages)
    out = [torch.empty_like(table), torch.empty_like(shares), free, i32([0, 0]),
           *(torch.empty(pages // 2, dtype=torch.int32, device="cuda") for _ in range(2))]
    lc.ar_pages_compact(i32(kv), table, shares, *out, scratch, page)
    want = S.compact(kv, table.tolist(), shares.tolist(), page, pages // 2)
    assert [out[i].tolist() for i in (0, 1, 3, 4, 5)] == list(want)
    assert out[2].tolist() == list(range(pages)) and not scratch.any()
    taken = want[2][0]
    gkv, gpool = torch.empty(nreq, dtype=torch.int32, device="cuda"), i32([0, 0])
    which = list(range(0, nreq, 3)) + [0, 5]
    lc.ar_pages_free(i32(which), i32(kv), out[0], out[1], out[3], out[2], gkv, gpool, scratch, page)
    shares, free, kv2, pool = S.free_pages(which, kv, want[0], want[1], [taken, pages], list(range(pages)), page)
    assert out[1].tolist() == shares and out[2].tolist() == free and gkv.tolist() == kv2 and gpool.tolist() == pool
    assert not scratch.any()


def test_state_that_does_not_hold_together(lc):
    """Pages freed more often than they were held, ids and pools out of range, rows longer than the table: what
    is written stays inside the buffers and scratch is left clean."""
    table = [[0, 0, 0, 1], [-1, 99, 2, 2 ** 31 - 1], [3, 4, 5, -2 ** 31], [1, 1, 1, 1]]
    shares, free = [0, 0, 5, -3, 0, 0], [9] * 6
    for pool in ([6, 6], [2, 6], [-4, 6], [100, 100]):
        for kv in ([64, 64, 64, 64], [2 ** 31 - 1, -5, 1, 0]):
            gs, gf, scratch = i32(shares), i32(free), lc.ar_pages_scratch(6)
            gk, gp = i32([7] * 4), i32([7, 7])
            lc.ar_pages_free(i32([0, 3, 1, 2, 2]), i32(kv), i32(table), gs, i32(pool), gf, gk, gp, scratch, 16)
            want = S.free_pages([0, 3, 1, 2, 2], kv, table, shares, pool, free, 16)
            assert (gs.tolist(), gf.tolist(), gk.tolist(), gp.tolist()) == want
            assert not scratch.any()
            t, so, mv = i32([[7] * 4] * 4), i32([7] * 6), [i32([7] * 3), i32([7] * 3)]
            lc.ar_pages_compact(i32(kv), i32(table), i32(shares), t, so, gf, gp, *mv, scratch, 16)
            want = S.compact(kv, table, shares, 16, 3)
            assert [t.tolist(), so.tolist(), gp.tolist(), mv[0].tolist(), mv[1].tolist()] == list(want)
            # forks of rows longer than the table are refused, invalid ids go along
            lists = [i32([7] * 3) for _ in range(3)]
            gt, gs = i32(table + [[-1] * 4] * 3), i32(shares)
            gk = i32([7] * 7)
            lc.ar_pages_fork(i32([0, 1, 2]), i32([4, 5, 6]), i32(kv + [0] * 3), gt, gs, i32(pool), i32(free), gk, gp, *lists, 16)
            want = S.fork([0, 1, 2], [4, 5, 6], kv + [0] * 3, table + [[-1] * 4] * 3, shares, pool, free, 16)
            assert [gt.tolist(), gs.tolist(), gk.tolist(), gp.tolist(), *(x.tolist() for x in lists)] == list(want)


def test_empty_lists(lc):
    s = State(lc, 3, 2, 10, 16)
    s.grow([5, 20, 0])
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    kv, pool = torch.empty_like(s.gkv), torch.empty_like(s.gpool)
    lc.ar_pages_fork(none, none, s.gkv, s.gtable, s.gshares, s.gpool, s.gfree, kv, pool, none, none, none, 16)
    assert kv.tolist() == s.kv and pool.tolist() == s.pool
    kv.zero_(), pool.zero_()
    lc.ar_pages_free(none, s.gkv, s.gtable, s.gshares, s.gpool, s.gfree, kv, pool, s.scratch, 16)
    assert kv.tolist() == s.kv and pool.tolist() == s.pool
    s.check()
    lc.ar_pages_copy([], none, none)
    lc.ar_pages_copy([s.gfree], none, none)


@pytest.mark.parametrize("shapes", [
    [(64,)], [(2, 3), (1,)], [(5, 7, 3)], [(4, 2, 16384), (4, 2, 2)], [(16384,), (16385,), (3, 16384)],
    [(8,)] * 130, [(100,), (4096,), (31,), (40000,)],
])
def test_copies(lc, shapes):
    """Pages of many sizes, in one call and more than one launch; ids out of range and pairs of one id skipped."""
    pages = 37
    g = torch.Generator(device="cuda")
    g.manual_seed(len(shapes))
    caches = [torch.randint(0, 256, (pages, *s), dtype=torch.uint8, device="cuda", generator=g) for s in shapes]
    before = [c.clone() for c in caches]
    src = [0, 5, -1, 7, 36, 9, 40, 3, 3, 2 ** 31 - 1]
    dst = [1, 6, 8, -1, 35, 9, 10, 20, 21, -2 ** 31]
    lc.ar_pages_copy(caches, i32(src), i32(dst))
    for c, b in zip(caches, before):
        for s, d in zip(src, dst):
            if 0 <= s < pages and 0 <= d < pages:
                b[d] = b[s]
        assert torch.equal(c, b)


def test_copies_of_other_types_and_unaligned_buffers(lc):
    whole = torch.arange(4096, dtype=torch.uint8, device="cuda")
    for off, shape in ((0, (16, 48)), (4, (16, 20)), (1, (16, 33)), (2, (16, 16))):
        n = shape[0] * shape[1]
        x = whole.clone()[off:off + n].view(shape)
        b = x.clone()
        lc.ar_pages_copy((x,), i32([1, 15]), i32([0, 14]))
        b[0], b[14] = b[1], b[15]
        assert torch.equal(x, b)
    for dtype in (torch.float32, torch.bfloat16, torch.int64):
        x = torch.arange(60, device="cuda").to(dtype).view(10, 6)
        b = x.clone()
        lc.ar_pages_copy([x], i32([9]), i32([4]))
        b[4] = b[9]
        assert torch.equal(x, b)


def test_long_lists_of_few_copies(lc):
    n = 20000
    x = torch.randint(0, 256, (n, 600), dtype=torch.uint8, device="cuda")
    b = x.clone()
    src, dst = (torch.full((n,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    at = torch.randperm(n // 2, device="cuda")[:500]
    src[at], dst[at] = at.int() + n // 2, at.int()
    src[-1], dst[-1] = n - 1, n // 2 - 1
    lc.ar_pages_copy([x, x[:, :4].contiguous()], src, dst)
    live = src >= 0
    b[dst[live].long()] = b[src[live].long()]
    assert torch.equal(x, b)


def test_pages_past_two_gigabytes(lc):
    x = torch.zeros(5, 1 << 29, dtype=torch.uint8, device="cuda")
    x[4, -100:], x[4, :100] = 3, 5
    lc.ar_pages_copy([x], i32([4]), i32([0]))
    assert torch.equal(x[0], x[4]) and not x[1:4].any()


def test_captured_and_replayed(lc):
    """Fork, copy and free captured as one graph, replayed with eager calls on the same scratch between."""
    page, pages, layers = 16, 40, 2
    s = State(lc, 6, 5, pages, page)
    s.grow([70, 37, 0, 0, 0, 0])
    caches = [torch.randint(0, 256, (pages, 64), dtype=torch.uint8, device="cuda") for _ in range(layers)]
    src, dst = i32([0, 1, 0]), i32([3, 4, 5])
    kv1, kv2 = torch.empty_like(s.gkv), torch.empty_like(s.gkv)
    pool1, pool2 = torch.empty_like(s.gpool), torch.empty_like(s.gpool)
    lists = [torch.empty(3, dtype=torch.int32, device="cuda") for _ in range(3)]

    def run():
        lc.ar_pages_fork(src, dst, s.gkv, s.gtable, s.gshares, s.gpool, s.gfree, kv1, pool1, *lists, page)
        lc.ar_pages_copy(caches, lists[0], lists[1])
        lc.ar_pages_free(dst, kv1, s.gtable, s.gshares, pool1, s.gfree, kv2, pool2, s.scratch, page)

    run()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    for i in range(3):
        for x in (kv1, kv2, pool1, pool2, *lists):
            x.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.tolist() for x in (kv1, kv2, pool1, pool2, *lists, s.gfree, s.gshares, s.gtable)]
        run()
        torch.cuda.synchronize()
        assert got == [x.tolist() for x in (kv1, kv2, pool1, pool2, *lists, s.gfree, s.gshares, s.gtable)], i
        assert kv2.tolist() == s.kv and pool2.tolist() == s.pool and not s.scratch.any() and not s.gshares.any()
        for c in caches:
            a, b = lists[0].long(), lists[1].long()
            assert torch.equal(c[a], c[b])


def test_buffers_on_the_host_or_of_other_sizes_are_refused(lc):
    x, n = torch.zeros(4, 8, device="cuda"), i32([0])
    with pytest.raises(ValueError, match="GPU"):
        lc.ar_pages_copy([x.cpu()], n, n)
    with pytest.raises(ValueError, match="same number of pages"):
        lc.ar_pages_copy([x, x[:3]], n, n)
    with pytest.raises(ValueError, match="contiguous"):
        lc.ar_pages_copy([x[:, ::2]], n, n)
    with pytest.raises(ValueError, match="dst"):
        lc.ar_pages_copy([x], i32([0, 1]), n)
    t = i32([[0, 0]])
    with pytest.raises(ValueError, match="scratch"):
        lc.ar_pages_free(n, n, t, i32([0] * 33), i32([0, 0]), n, i32([0]), i32([0, 0]), i32([0, 0]), 16)
    with pytest.raises(ValueError, match="table_out"):
        lc.ar_pages_compact(n, t, i32([0, 0]), i32([[0]]), i32([0, 0]), i32([0, 0]), i32([0, 0]), i32([0]), i32([0]), i32([0, 0]), 16)
