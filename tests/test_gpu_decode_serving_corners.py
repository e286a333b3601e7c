"""Calls of the serving operators that their documentation allows, at their corners: graphs of the forms for many rows and of
the compaction, two handles on two streams, one slot twice, padding between and behind large prompts, pools at the size
where the compaction's LDS passes 64 KiB."""

import math
import random

import pytest
import torch

from tests import serving_ref as S
from tests.test_gpu_decode_attention_forms import compare, lc  # noqa: F401  (lc is the fixture)
from tests.test_gpu_decode_kv8_tiles import Batch
from tests.test_gpu_decode_pages import State, i32

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("d,size", [(128, (24, 190, 900)), (64, (24, 190, 900)), (96, (24, 64, 900)), (192, (24, 24, 500)), (128, (24, 24, 500))])
def test_chunks_captured_and_replayed(lc, d, size):  # noqa: F811
    """One captured call over changing lengths, queries and starts, with eager calls on the same handle between."""
    c = Batch(lc, d, *size)
    kv, starts = i32(c.kv), i32(c.starts)
    out, lse = torch.full_like(c.q, 7.0), torch.full(c.q.shape[:2], 7.0, device="cuda")

    def call():
        lc.ar_kv8_attention(c.h, c.q, c.data, c.scales, c.table, kv, starts, out, lse, 0.02, 0)

    call()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    t = c.starts[-1]
    for i in range(4):
        kv.copy_(torch.tensor([max(n - 97 * i, 0) for n in c.kv], dtype=torch.int32))
        starts.copy_(torch.tensor([min(s + 11 * i, t) for s in c.starts], dtype=torch.int32))
        c.q.normal_()
        out.fill_(7.0), lse.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got, got_lse = out.clone(), lse.clone()
        out.fill_(7.0), lse.fill_(7.0)
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, got) and torch.equal(lse, got_lse), i
        assert (out[:11 * i] == 7).all() and (out[11 * i:] != 7).any()
    c.done()


def test_two_handles_on_two_streams(lc):  # noqa: F811
    """Chunks of two batches at once, each with a handle of its own: the bits that each gives alone."""
    a, b = Batch(lc, 128, 24, 190, 900, seed=1), Batch(lc, 96, 24, 64, 900, seed=2)
    want = [c.call() for c in (a, b)]
    outs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    args = [(c, i32(c.kv), i32(c.starts), torch.empty_like(c.q), torch.empty(c.q.shape[:2], device="cuda")) for c in (a, b)]
    torch.cuda.synchronize()
    for s, (c, kv, starts, out, lse) in zip(streams, args):
        with torch.cuda.stream(s):
            for _ in range(6):
                lc.ar_kv8_attention(c.h, c.q, c.data, c.scales, c.table, kv, starts, out, lse, 0.02, 0)
        outs.append((out, lse))
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    a.done(), b.done()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128, 192])
def test_large_prompts_among_tokens_of_nobody(lc, dtype, d):  # noqa: F811
    """NaN and infinities before, between and behind prompts of many rows; their rows stay."""
    starts, hq, hkv = [70, 70, 1000, 1001, 1400], 64, 4  # the call's first 70 and last 133 tokens are nobody's
    t = 1533
    g = torch.Generator(device="cuda").manual_seed(d)
    q, k, v = (torch.randn(t, n, d, generator=g, device="cuda").to(dtype) for n in (hq, hkv, hkv))
    for x, bad in ((q, math.nan), (k, math.nan), (v, math.inf)):
        x[:70], x[1400:] = bad, bad
    h = lc.ar_prompt_create(hkv, d)
    for window in (0, 200):
        out, lse = torch.full_like(q, 7.0), torch.full((t, hq), 7.0, device="cuda")
        lc.ar_prompt_attention(h, q, k, v, i32(starts), out, lse, None, window)
        torch.cuda.synchronize()
        for a, b in ((70, 1000), (1000, 1001), (1001, 1400)):
            compare(out[a:b], lse[a:b], S.dense_attention(q[a:b], k[a:b], v[a:b], d ** -0.5, window))
        for x in (out, lse):
            assert (x[:70] == 7).all() and (x[1400:] == 7).all()
    lc.ar_prompt_destroy(h)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_slot_twice_leaves_the_other_blocks_right(lc, dtype):  # noqa: F811
    """Two tokens with one slot, and tokens in another order: those blocks are undefined, every other is as it would be."""
    heads, d, page, pages = 3, 128, 32, 6
    h = lc.ar_kv8_create(heads, d, page)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(90, heads, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    slots = torch.arange(90, device="cuda")
    clean = lc.ar_kv8_cache(h, pages)
    lc.ar_kv8_append(h, k, v, slots, *clean)
    twice = slots.clone()
    twice[20] = 18          # block 1
    twice[40:44] = twice[40:44].flip(0)  # block 2, backwards
    twice[70] = 69          # block 4
    got = lc.ar_kv8_cache(h, pages)
    lc.ar_kv8_append(h, k, v, twice, *got)
    torch.cuda.synchronize()
    (x, _), (y, _) = (S.unpack(c[0].cpu(), c[1].cpu(), d) for c in (clean, got))  # [pages, heads, 2, page, d]
    x, y = (z.permute(0, 3, 1, 2, 4).reshape(pages * page // 16, 16, heads, 2, d) for z in (x, y))
    for block in range(pages * page // 16):
        if block not in (1, 2, 4):
            assert torch.equal(x[block], y[block]), block
    lc.ar_kv8_destroy(h)


@pytest.mark.parametrize("pages", [262080, 262112, 262113, 262144])
def test_compaction_where_its_lds_passes_64_kib(lc, pages):  # noqa: F811
    nreq, width, page = 16, 512, 16
    rng = random.Random(pages)
    table = torch.randperm(pages, device="cuda")[:nreq * width].view(nreq, width).int()
    kv = [rng.randrange(0, width * page + 1) for _ in range(nreq)]
    shares, free = torch.zeros(pages, dtype=torch.int32, device="cuda"), torch.empty(pages, dtype=torch.int32, device="cuda")
    out = [torch.empty_like(table), torch.empty_like(shares), free, i32([0, 0]),
           *(torch.empty(pages // 2, dtype=torch.int32, device="cuda") for _ in range(2))]
    scratch = lc.ar_pages_scratch(pages)
    lc.ar_pages_compact(i32(kv), table, shares, *out, scratch, page)
    want = S.compact(kv, table.tolist(), shares.tolist(), page, pages // 2)
    assert [out[i].tolist() for i in (0, 1, 3, 4, 5)] == list(want)
    assert out[2].tolist() == list(range(pages)) and not scratch.any()


def test_compaction_captured_and_replayed(lc):  # noqa: F811
    """A compaction with its copies as one graph, over lengths that change; eager calls on the same scratch between."""
    page, pages, nreq, width = 16, 60, 5, 8
    s = State(lc, nreq, width, pages, page)
    s.grow([100, 37, 128, 1, 64])
    caches = [torch.randint(0, 256, (pages, 2, 48), dtype=torch.uint8, device="cuda") for _ in range(3)]
    table, shares = torch.empty_like(s.gtable), torch.empty_like(s.gshares)
    free, pool, kv = torch.empty_like(s.gfree), torch.empty_like(s.gpool), s.gkv.clone()
    moves = [torch.empty(pages // 2, dtype=torch.int32, device="cuda") for _ in range(2)]
    work = [c.clone() for c in caches]

    def run():
        for w, c in zip(work, caches):
            w.copy_(c)
        lc.ar_pages_compact(kv, s.gtable, s.gshares, table, shares, free, pool, *moves, s.scratch, page)
        lc.ar_pages_copy(work, *moves)

    run()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    for i in range(4):
        lens = [max(n - 30 * i, 0) for n in s.kv]
        kv.copy_(torch.tensor(lens, dtype=torch.int32))
        for x in (table, shares, free, pool, *moves):
            x.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.tolist() for x in (table, shares, pool, *moves)]
        assert got == list(S.compact(lens, s.table, s.shares, page, pages // 2)) and not s.scratch.any(), i
        for c, w in zip(caches, work):  # every held page is where its new id says
            for b in range(nreq):
                for j in range(S.pages_for(lens[b], page)):
                    assert torch.equal(w[got[0][b][j]], c[s.table[b][j]])
        run()
        torch.cuda.synchronize()
        assert got == [x.tolist() for x in (table, shares, pool, *moves)]


@pytest.mark.parametrize("d,size", [(64, (24, 24, 500)), (64, (24, 190, 900)), (96, (24, 64, 900)), (128, (24, 64, 900)), (128, (24, 190, 900)),
                                    (192, (24, 24, 500)), (256, (24, 64, 900)), (128, (24, 3, 500))])
def test_chunks_that_overlap_beside_ones_that_do_not(lc, d, size):  # noqa: F811
    """Starts that go back and forth: eleven requests over the same tokens. The first and the last are alone, and right."""
    c = Batch(lc, d, *size)
    t, first, last = c.starts[-1], c.new[0], max(c.new[-1], 1)
    c.starts = [0, first] + [t - last, first] * 11 + [t]
    c.starts[-2] = t - last
    c.new = [max(b - a, 0) for a, b in zip(c.starts, c.starts[1:])]
    out, lse = c.call()
    values = S.unpack(c.data.cpu(), c.scales.cpu(), d)[0].cuda()
    for b in (0, 23):
        m, n = c.new[b], c.kv[b]
        kv = values[c.table[b].long()].permute(2, 0, 3, 1, 4).reshape(2, -1, c.hkv, d)[:, :n]
        a = slice(c.starts[b], c.starts[b + 1])
        assert 0 < m <= n
        compare(out[a], lse[a], S.dense_attention(c.q[a], kv[0], kv[1], 0.02, 0))
    assert (lse[first:t - last] != 7).all()
    c.done()
