"""Rows into and out of the 8-bit cache on the GPU against the plain form (serving_ref.Cache): the values that
the cache stands for and its scales are equal, not near; the joined form against its parts."""

import math

import pytest
import torch

from tests import serving_ref as S

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lc():
    import latency_collectives_amd as lc

    return lc


class Pool:
    """A cache on the GPU beside its plain form."""

    def __init__(self, lc, pages, heads, d, page, dtype):
        self.lc, self.d, self.page, self.dtype, self.pages, self.heads = lc, d, page, dtype, pages, heads
        self.h = lc.ar_kv8_create(heads, d, page)
        self.data, self.scales = lc.ar_kv8_cache(self.h, pages)
        self.ref = S.Cache(pages, heads, d, page)
        self.written = torch.zeros(pages * page, dtype=torch.bool)

    def append(self, k, v, slots):
        """k, v [T, heads, D] on the CPU, of the pool's type."""
        t = len(slots)
        # strided as the projection's output is
        both = torch.cat([k.reshape(t, -1), v.reshape(t, -1)], dim=1).cuda()
        kk, vv = (x.view(t, self.heads, self.d) for x in both.split(self.heads * self.d, dim=1))
        self.lc.ar_kv8_append(self.h, kk, vv, torch.tensor(slots, dtype=torch.int64, device="cuda"), self.data, self.scales)
        self.ref.append(k, v, slots)
        for s in slots:
            if 0 <= s < self.pages * self.page:
                if s % 16 == 0:
                    self.written[s:s + 16] = False  # a block that begins afresh
                self.written[s] = True

    def check(self):
        values, e = S.unpack(self.data.cpu(), self.scales.cpu(), self.d)
        live = self.written.view(self.pages, self.page)
        got = values.permute(0, 3, 1, 2, 4)[live]
        want = self.ref.values.permute(0, 3, 1, 2, 4)[live]
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))
        blocks = live.view(self.pages, -1, 16).any(-1)
        assert torch.equal(e.transpose(1, 2)[blocks], self.ref.e.transpose(1, 2)[blocks])
        # and read back
        slots = torch.nonzero(self.written).flatten()
        slots = torch.cat([slots, torch.tensor([-1, self.pages * self.page])]).cuda()
        k, v = (torch.full((slots.numel(), self.heads, self.d), 9.0, dtype=BF, device="cuda") for _ in range(2))
        self.lc.ar_kv8_read(self.h, slots, self.data, self.scales, k, v)
        back = torch.stack([k, v], dim=2).cpu().double()
        assert torch.equal(back[:-2].nan_to_num(nan=7.0), want.nan_to_num(nan=7.0)) and (back[-2:] == 0).all()

    def done(self):
        torch.cuda.synchronize()
        self.lc.ar_kv8_destroy(self.h)


def rows(g, t, heads, d, dtype, spread=2.0):
    size = torch.exp(spread * torch.randn(t, heads, 1, generator=g))
    return [(torch.randn(t, heads, d, generator=g) * size).to(dtype) for _ in range(2)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("heads,page", [(1, 16), (3, 64)])
def test_prompts_then_single_tokens(lc, dtype, d, heads, page):
    """Requests' prompts, chunks that begin inside a block, then single tokens whose size grows and falls."""
    g = torch.Generator().manual_seed(d + page)
    pool = Pool(lc, 14, heads, d, page, dtype)
    ids = torch.randperm(14, generator=g).tolist()
    lens, room = [0, 0, 0], 4 * page
    pages = [ids[4 * b:4 * b + 4] for b in range(3)]

    def step(new):
        slots = []
        for b, n in enumerate(new):
            slots += [pages[b][i // page] * page + i % page for i in range(lens[b], lens[b] + n)]
            lens[b] += n
        k, v = rows(g, len(slots), heads, d, dtype)
        pool.append(k, v, slots)

    step([17, 1, 33])
    pool.check()
    step([3, 20, 0])
    step([room - 30, 5, 7 if page == 16 else 50])
    pool.check()
    for _ in range(9):
        step([1, 1, 1])
    pool.check()
    pool.done()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_tokens_at_once(lc, dtype):
    """More runs than are looked for one by one: a wave finds them in windows of 16 tokens, of prompts that
    begin anywhere, single tokens, and slots that are nowhere."""
    g = torch.Generator().manual_seed(5)
    heads, d, page, pages = 4, 64, 32, 100
    pool = Pool(lc, pages, heads, d, page, dtype)
    slots, at = [], 0
    while at < pages * page - 300:
        n = int(torch.randint(1, 100, (1,), generator=g))
        slots += list(range(at, at + n)) + [-1] * int(torch.randint(0, 3, (1,), generator=g))
        at = (at + n + 15) // 16 * 16 + 16 * int(torch.randint(0, 2, (1,), generator=g))
    assert len(slots) * heads * 2 >= 16384
    k, v = rows(g, len(slots), heads, d, dtype)
    pool.append(k, v, slots)
    pool.check()
    pool.done()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_special_values(lc, dtype):
    """Zeros, the largest and the smallest numbers, infinities and NaN, in fresh blocks and beside others."""
    big = torch.finfo(dtype).max
    for first in ([0.0], [1.0], [big], [1e-38], [math.inf, 1.0], [math.nan, 3.0]):
        for then in (0.0, -0.0, 2.0 ** -110, 448.0, 449.0, -big, math.inf, -math.inf, math.nan, 2.0 ** -126):
            pool = Pool(lc, 1, 1, 64, 16, dtype)
            x = torch.ones(len(first) + 1, 1, 64)
            x[:len(first), 0] = torch.tensor(first)[:, None]
            x[0, 0, 5] = 0.25
            pool.append(x[:len(first)].to(dtype), (-x[:len(first)]).to(dtype), list(range(len(first))))
            x[-1, 0, ::3] = then
            pool.append(x[-1:].to(dtype), (-x[-1:]).to(dtype), [len(first)])
            pool.check()
            pool.done()


def test_scales_at_their_borders(lc):
    """Largest elements of 448 times a power of two and one step to either side."""
    for dtype, step in ((F32, 2.0 ** -23), (BF, 2.0 ** -7)):
        for e in (-100, -99, -20, 0, 7, 118, 119):
            for f in (1 - step, 1.0, 1 + step):
                pool = Pool(lc, 1, 1, 64, 16, dtype)
                x = torch.full((1, 1, 64), 448.0 * f) * 2.0 ** e
                pool.append(x.to(dtype), (x / 2).to(dtype), [0])
                pool.check()
                pool.done()


def test_slots_that_are_nowhere_write_nothing(lc):
    pool = Pool(lc, 3, 2, 96, 16, F32)
    g = torch.Generator().manual_seed(1)
    k, v = rows(g, 7, 2, 96, F32)
    pool.data.fill_(0x55), pool.scales.fill_(0x66)
    before = pool.data.clone(), pool.scales.clone()
    slots = torch.tensor([-1, 48, 2 ** 40, -2 ** 40, 2 ** 62, -2 ** 63, 49], device="cuda")
    lc.ar_kv8_append(pool.h, k.cuda(), v.cuda(), slots, pool.data, pool.scales)
    assert torch.equal(pool.data, before[0]) and torch.equal(pool.scales, before[1])
    # one row: its block, and no other
    slots[3] = 16
    lc.ar_kv8_append(pool.h, k.cuda(), v.cuda(), slots, pool.data, pool.scales)
    assert torch.equal(pool.data[[0, 2]], before[0][[0, 2]]) and torch.equal(pool.scales[[0, 2]], before[1][[0, 2]])
    assert not torch.equal(pool.data[1], before[0][1])
    pool.done()


def test_rows_behind_a_single_token_stay(lc):
    """A token inside a block changes its own row alone where the scale holds, whatever lies behind it."""
    pool = Pool(lc, 1, 1, 128, 16, BF)
    pool.append(*[torch.full((1, 1, 128), 100.0, dtype=BF)] * 2, [0])
    pool.data.view(-1)[:] = torch.where(pool.data.view(-1) == 0, 0x7F, pool.data.view(-1))
    k0, _ = pool.data[0, 0, 0].clone(), pool.data[0, 0, 1].clone()
    pool.append(*[torch.full((1, 1, 128), 3.0, dtype=BF)] * 2, [1])
    pool.check()
    k1 = pool.data[0, 0, 0].view(16, 128)
    assert torch.equal(k1[2:], k0.view(16, 128)[2:]) and torch.equal(k1[0], k0.view(16, 128)[0])
    pool.done()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (96, 48, True), (128, 128, False), (192, 96, False),
                                         (256, 256, True), (128, 0, False)])
@pytest.mark.parametrize("normed", [True, False])
def test_joined_with_norm_and_rotation(lc, dtype, d, rot, inter, normed):
    """The same bits as the norm and rotation followed by the append, padding and refused tokens among them."""
    g = torch.Generator().manual_seed(d + rot)
    for hq, hkv, t in ((3, 2, 21), (8, 1, 1), (0, 2, 5), (16, 8, 1100)):
        page, pages = 32, 80
        h = lc.ar_kv8_create(hkv, d, page)
        a, b = lc.ar_kv8_cache(h, pages), lc.ar_kv8_cache(h, pages)
        qkv = torch.randn(t, (hq + 2 * hkv) * d, generator=g).to(dtype).cuda()
        q, k, v = (x.view(t, n, d) for x, n in zip(qkv.split([hq * d, hkv * d, hkv * d], dim=1), (hq, hkv, hkv)))
        angle = torch.randn(64, max(rot // 2, 1), generator=g)
        cs = torch.cat([angle.cos(), angle.sin()], dim=1).cuda() if rot else None
        # a position past the table's end is NaN; below zero, padding
        positions = torch.arange(t) % 66
        positions[3::11] = -1
        positions = positions.int().cuda()
        slots = (torch.arange(t) + 5).cuda()
        slots[t // 2] = -1
        w = [(1 + 0.1 * torch.randn(d, generator=g)).to(dtype).cuda() for _ in range(2)] if normed else [None, None]
        q1, q2, k2 = torch.full_like(q, 7.0), torch.full_like(q, 7.0), torch.zeros_like(k)
        lc.ar_kv8_norm_rope_append(h, q, k, v, q1, positions, cs, slots, *a, *w, 1e-5, inter)
        lc.ar_qk_norm_rope(q, k, q2, k2, positions, cs, *w, 1e-5, inter)
        lc.ar_kv8_append(h, k2, v, torch.where(positions < 0, -1, slots), *b)
        # the values: a rotated NaN may carry another sign
        assert torch.equal(q1.view(torch.int16 if dtype == BF else torch.int32),
                           q2.view(torch.int16 if dtype == BF else torch.int32))
        x, ex = S.unpack(a[0].cpu(), a[1].cpu(), d)
        y, ey = S.unpack(b[0].cpu(), b[1].cpu(), d)
        assert torch.equal(torch.isnan(x), torch.isnan(y)) and torch.equal(x.nan_to_num(), y.nan_to_num())
        assert torch.equal(ex, ey)
        torch.cuda.synchronize()
        lc.ar_kv8_destroy(h)


def test_captured_and_on_another_stream(lc):
    """A captured step replayed over new inputs, and a call on a side stream, against eager calls."""
    heads, d, page, pages = 2, 128, 16, 6
    h = lc.ar_kv8_create(heads, d, page)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    k, v = (torch.randn(4, heads, d, device="cuda", generator=g) for _ in range(2))
    slots = torch.tensor([0, 17, 40, 64], device="cuda")
    cache, want = lc.ar_kv8_cache(h, pages), lc.ar_kv8_cache(h, pages)
    lc.ar_kv8_append(h, k, v, slots, *cache)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            lc.ar_kv8_append(h, k, v, slots, *cache)
    lc.ar_kv8_append(h, k, v, slots, *want)
    for i in range(4):
        k.normal_(generator=g), v.normal_(generator=g)
        slots += 1
        torch.cuda.synchronize()
        graph.replay()
        lc.ar_kv8_append(h, k, v, slots, *want)
        torch.cuda.synchronize()
        assert torch.equal(cache[0], want[0]) and torch.equal(cache[1], want[1]), i
    with torch.cuda.stream(side):
        lc.ar_kv8_append(h, k, v, slots + 1, *cache)
    lc.ar_kv8_append(h, k, v, slots + 1, *want, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(cache[0], want[0])
    lc.ar_kv8_destroy(h)


def test_tensors_that_want_gradients_are_refused(lc):
    h = lc.ar_kv8_create(2, 64, 16)
    cache = lc.ar_kv8_cache(h, 1)
    k = torch.zeros(1, 2, 64, device="cuda", requires_grad=True)
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="gradient"):
        lc.ar_kv8_append(h, k, k, slots, *cache)
    with torch.no_grad():
        lc.ar_kv8_append(h, k, k, slots, *cache)
    torch.cuda.synchronize()
    lc.ar_kv8_destroy(h)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_most_tokens_at_once(lc, dtype):
    """As test_many_tokens_at_once, where a wave looks for runs in 16 tokens."""
    g = torch.Generator().manual_seed(6)
    heads, d, page, pages = 12, 64, 32, 100
    pool = Pool(lc, pages, heads, d, page, dtype)
    slots, at = [], 0
    while at < pages * page - 120:
        n = int(torch.randint(1, 100, (1,), generator=g))
        slots += list(range(at, at + n)) + [-1] * int(torch.randint(0, 3, (1,), generator=g))
        at = (at + n + 15) // 16 * 16
    slots += [-1] * max(0, 65536 // (2 * heads) + 1 - len(slots))
    assert len(slots) * heads * 2 >= 65536
    k, v = rows(g, len(slots), heads, d, dtype)
    pool.append(k, v, slots)
    pool.check()
    pool.done()


@pytest.mark.parametrize("tokens", [1400, 11003])
@pytest.mark.parametrize("prompts", [True, False])
def test_many_tokens_joined_with_norm_and_rotation(lc, tokens, prompts):
    """Runs of up to 16 tokens and of one, in windows of 4 and of 16: what the parts give, to the bit."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    heads, d, page = 3, 64, 64
    h = lc.ar_kv8_create(heads, d, page)
    pages = (tokens if prompts else tokens * 16) // page + 2
    q, k, v = (torch.randn(tokens, n, d, generator=g, device="cuda").bfloat16() for n in (6, heads, heads))
    at = torch.arange(tokens, device="cuda") if prompts else torch.randperm(tokens, generator=g, device="cuda") * 16 + 5
    positions = (torch.arange(tokens, device="cuda") % 500).int()
    positions[torch.randperm(tokens, generator=g, device="cuda")[:tokens // 20]] = -1
    cs = torch.randn(500, d, generator=g, device="cuda")
    w = torch.randn(d, generator=g, device="cuda").bfloat16()
    one, two = (lc.ar_kv8_cache(h, pages) for _ in range(2))
    q1, q2, k2 = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(k)
    lc.ar_kv8_norm_rope_append(h, q, k, v, q1, positions, cs, at, *one, w, w)
    lc.ar_qk_norm_rope(q, k, q2, k2, positions, cs, w, w)
    lc.ar_kv8_append(h, k2, v, torch.where(positions < 0, -1, at), *two)
    torch.cuda.synchronize()
    assert torch.equal(q1, q2) and torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    assert (one[1] != 0).any()
    lc.ar_kv8_destroy(h)
