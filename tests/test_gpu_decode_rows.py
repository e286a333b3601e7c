"""ar_page_tables, ar_qk_norm_rope and the 4-bit cache's rows on the GPU against the plain 64-bit
forms of decode_ref. Integers and stored codes are equal; a rotated value is one rounding of a
64-bit value, so it is within half a step (and half a binary32 step, which it passes through)."""

import pytest
import torch

from tests import decode_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lc():
    import latency_collectives_amd as lc

    return lc


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ page tables


def _run_tables(lc, cached, new, pool, free, table, ntokens, page, stride=None):
    n = len(cached)
    width = len(table[0]) if n else 3
    buf = torch.full((max(n, 1), stride or width), -7, dtype=torch.int32, device="cuda")
    if n:
        buf[:, :width] = _i32(table)
    out = dict(kv=_i32([-9] * max(n, 1)), q=_i32([-9] * (n + 1)),
               slots=torch.full((ntokens,), -9, dtype=torch.int64, device="cuda"),
               pos=torch.full((ntokens,), -9, dtype=torch.int32, device="cuda"),
               pool=_i32([-9, -9]), refused=_i32([-9] * max(n, 1)))
    args = (_i32(cached), _i32(new), _i32(pool), _i32(free), buf[:n, :width] if n else buf[:, :width],
            out["kv"][:n], out["q"], out["slots"], out["pos"], out["pool"], out["refused"][:n], page)
    for _ in range(2):  # inputs are only read: a second call gives the same
        lc.ar_page_tables(*args)
    torch.cuda.synchronize()
    if stride:
        assert (buf[:, width:] == -7).all()
    return (buf[:n, :width].tolist(), out["kv"][:n].tolist(), out["q"].tolist(), out["slots"].tolist(),
            out["pos"].tolist(), out["pool"].tolist(), out["refused"][:n].tolist())


def _case(seed, n, page, most_cached, most_new, short=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    cached = torch.randint(0, most_cached + 1, (n,), generator=g).tolist()
    new = torch.randint(0, most_new + 1, (n,), generator=g).tolist()
    width = max(1, max(-(-(c + m) // page) for c, m in zip(cached, new)))
    held = [-(-c // page) for c in cached]
    need = sum(-(-(c + m) // page) for c, m in zip(cached, new)) - sum(held)
    ids = torch.randperm(sum(held) + need + 11, generator=g).tolist()
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    free = ids[at:]
    head = 3
    return cached, new, [head, head + max(0, need - short)], [0] * head + free, table, sum(new) + pad, page


@pytest.mark.parametrize("n,page,cached,new,pad", [
    (1, 16, 0, 1, 0), (1, 16, 15, 1, 3), (3, 1, 9, 4, 0), (64, 16, 300, 1, 5), (65, 32, 100, 40, 1),
    (1023, 16, 500, 2, 0), (1025, 7, 60, 3, 9), (4096, 64, 2000, 6, 100), (5, 128, 4000, 9000, 0),
])
def test_page_tables(lc, n, page, cached, new, pad):
    case = _case(n + page, n, page, cached, new, 0, pad)
    assert _run_tables(lc, *case, stride=len(case[4][0]) + 3) == tuple(R.page_tables(*case))


@pytest.mark.parametrize("short", [1, 7, 10 ** 6])
def test_page_tables_with_too_few_pages(lc, short):
    case = _case(5, 200, 16, 100, 30, short, 4)
    want = R.page_tables(*case)
    assert sum(want[6]) > 0
    assert _run_tables(lc, *case) == tuple(want)


def test_page_tables_refusals_on_the_device(lc):
    """Negative lengths, a row that is too short, too few token places, a negative page id, a
    free list whose end lies beyond its entries; no request at all."""
    case = ([5, -1, 3, 30, 4, 2 ** 31 - 5], [1, 2, -3, 9, 2, 20], [0, 99], [4, 5, 6], [[9, -1], [1, 1], [2, 2], [3, 7], [-5, -1], [6, 6]], 64, 16)
    assert _run_tables(lc, *case) == tuple(R.page_tables(*case))
    case = ([0, 0, 0], [5, 6, 7], [0, 8], list(range(8)), [[-1], [-1], [-1]], 12, 16)
    got = _run_tables(lc, *case)
    assert got == tuple(R.page_tables(*case)) and got[6] == [0, 0, 1]
    got = _run_tables(lc, [], [], [2, 5], [1, 2, 3, 4, 5], [], 3, 16)
    assert got[2:6] == ([0], [-1, -1, -1], [-1, -1, -1], [2, 5])


def test_page_tables_steps_follow_each_other(lc):
    """Lengths and the pool of one step are those of the next, without the host in between."""
    page, n, steps = 16, 5, 40
    cached, free = [0, 15, 16, 31, 7], list(range(100, 140))
    table = [[90 + 3 * b + j if j < -(-c // page) else -1 for j in range(6)] for b, c in enumerate(cached)]
    kv = [_i32(cached), _i32([0] * n)]
    pool = [_i32([0, 40]), _i32([0, 0])]
    buf, one = _i32(table), _i32([1] * n)
    want_cached, want_pool, want_table = cached, [0, 40], table
    for s in range(steps):
        slots = torch.empty(n, dtype=torch.int64, device="cuda")
        pos, q, ref = _i32([0] * n), _i32([0] * (n + 1)), _i32([0] * n)
        lc.ar_page_tables(kv[s % 2], one, pool[s % 2], _i32(free), buf, kv[1 - s % 2], q, slots, pos,
                          pool[1 - s % 2], ref, page)
        want = R.page_tables(want_cached, [1] * n, want_pool, free, want_table, n, page)
        want_table, want_cached, want_pool = want[0], want[1], want[5]
        assert slots.tolist() == want[3] and buf.tolist() == want_table


# ------------------------------------------------------------------ norm and rotation


def _cos_sin(rows, rot):
    a = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2).double() / rot)
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _close(got, want, dtype, scale):
    """Within one rounding of the 64-bit value: half a step of the type, half a binary32 step on
    the way, 2^-48 of the terms for the 64-bit arithmetic and the type's smallest step."""
    tiny = 2.0 ** -133 if dtype == BF else 2.0 ** -149
    bound = (R.HALF[dtype] + 2.0 ** -24) * want.abs() + 2.0 ** -48 * scale + tiny
    got = got.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    err = torch.where(torch.isnan(want), 0.0, (got - want).abs())
    bound = torch.where(torch.isnan(want), 0.0, bound)
    assert (err <= bound).all(), float((err - bound).max())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t,hq,hkv,d,rot,inter,weights", [
    (1, 1, 1, 64, 64, False, True), (1, 8, 1, 128, 128, False, True), (5, 3, 1, 96, 96, True, True),
    (17, 4, 4, 128, 64, False, True), (33, 7, 2, 192, 192, False, False), (9, 5, 5, 256, 256, True, True),
    (3, 2, 1, 8, 8, False, True), (11, 6, 2, 40, 16, True, True), (4, 3, 3, 72, 0, False, True),
    (130, 12, 4, 248, 248, False, True), (2, 0, 3, 128, 128, False, True), (2, 3, 0, 128, 128, False, True),
])
def test_norm_rope(lc, dtype, t, hq, hkv, d, rot, inter, weights):
    g = torch.Generator().manual_seed(t * 7 + d)
    qkv = torch.randn(t, (hq + 2 * hkv) * d, generator=g).to(dtype)
    pos = torch.randint(0, 100, (t,), generator=g).int()
    cs = _cos_sin(100, rot) if rot else None
    wq, wk = ((1 + torch.randn(d, generator=g) / 4).to(dtype) for _ in range(2)) if weights else (None, None)
    dev = qkv.cuda()  # a packed projection: strided views
    q, k, _ = (x.view(t, -1, d) for x in dev.split([hq * d, hkv * d, hkv * d], dim=1))
    q_out = torch.full((t, hq + 1, d), 7.0, dtype=dtype, device="cuda")
    k_out = torch.full((t, hkv, d), 7.0, dtype=dtype, device="cuda")
    cu = lambda x: None if x is None else x.cuda()  # noqa: E731
    lc.ar_qk_norm_rope(q, k, q_out[:, :hq], k_out, cu(pos) if rot else None, cu(cs), cu(wq), cu(wk), 1e-5, inter)
    assert (q_out[:, hq] == 7.0).all()
    for got, x, w in ((q_out[:, :hq], q, wq), (k_out, k, wk)):
        if x.numel() == 0:
            continue
        want = R.norm_rope(x.cpu(), w, cs, pos, 1e-5, inter)
        _close(got, want, dtype, 64.0)
    # in place
    lc.ar_qk_norm_rope(q, k, q, k, cu(pos) if rot else None, cu(cs), cu(wq), cu(wk), 1e-5, inter)
    assert torch.equal(q, q_out[:, :hq]) and torch.equal(k, k_out)


def test_norm_rope_padding_far_positions_and_extremes(lc):
    """Negative positions write nothing, positions beyond the table give NaN, a zero row stays
    zero, an infinity or NaN stays in its own row, large and tiny values keep their norm."""
    t, d = 9, 128
    g = torch.Generator().manual_seed(3)
    x = torch.randn(t, 2, d, generator=g)
    x[2] = 0.0
    x[3, 0, 5], x[3, 1, 7] = float("inf"), float("nan")
    x[4] *= 1e30
    x[5] *= 1e-30
    pos = torch.tensor([0, -1, 3, 4, 5, 6, 50, 2 ** 31 - 1, 49]).int()
    cs = _cos_sin(50, d)
    w = torch.ones(d)
    for dtype in (BF, F32):
        q = x.to(dtype)
        out = torch.full((t, 2, d), 7.0, dtype=dtype, device="cuda")
        k_out = out.clone()
        lc.ar_qk_norm_rope(q.cuda(), q.cuda(), out, k_out, pos.cuda(), cs.cuda(), w.to(dtype).cuda(), None, 1e-6)
        assert (out[1] == 7.0).all() and (k_out[1] == 7.0).all()
        keep = [0, 2, 3, 4, 5, 6, 7, 8]
        want = R.norm_rope(q, w, cs, pos, 1e-6, False)[keep]
        _close(out[keep], want, dtype, 64.0)
        assert torch.isnan(out[6:8]).all() and torch.isnan(k_out[6:8]).all()
        assert (out[2] == 0).all() and torch.isfinite(out[[0, 2, 4, 5, 8]].float()).all()


# ------------------------------------------------------------------ the 4-bit cache


def _empty(lc, h, pages):
    data, scales = lc.ar_kv4_cache(h, pages)
    data.fill_(0xA5), scales.fill_(0xFF)
    return data, scales


def _reference_cache(data, scales, k, v, slots, page):
    data, scales = data.cpu().clone(), scales.cpu().clone()
    for which, x in ((0, k), (1, v)):
        code, sc = R.quantise(x.float().cpu())
        for t, s in enumerate(slots):
            if 0 <= s < data.shape[0] * page:
                for h in range(x.shape[1]):
                    R.pack_row(data, scales, page, s, h, which, code[t, h], sc[t, h])
    return data, scales


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t,heads,d,page", [(1, 1, 128, 16), (5, 3, 64, 16), (18, 2, 96, 32), (3, 1, 192, 1024),
                                            (40, 5, 256, 64), (33, 8, 128, 16)])
def test_append_and_read(lc, dtype, t, heads, d, page):
    g = torch.Generator().manual_seed(t + d)
    kv = torch.randn(t, 2 * heads * d, generator=g).to(dtype)
    kv *= torch.exp2(torch.randint(-12, 12, (t, 1), generator=g).float()).to(dtype)
    kv[0, :5] = torch.tensor([0.25, 2.5, -0.0, 3.5, 5.0]).to(dtype)
    k, v = (x.view(t, heads, d) for x in kv.cuda().split(heads * d, dim=1))
    pages = -(-t // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:t]
    if t > 4:
        slots[2], slots[3], slots[4] = -1, pages * page, 2 ** 40
    h = lc.ar_kv4_create(heads, d, page)
    data, scales = _empty(lc, h, pages)
    want = _reference_cache(data, scales, k, v, slots.tolist(), page)
    lc.ar_kv4_append(h, k, v, slots.cuda(), data, scales)
    assert torch.equal(scales.cpu(), want[1])
    assert torch.equal(data.cpu(), want[0])
    kk, vv = R.unpack(data.cpu(), scales.cpu(), page)
    for out_type in (BF, F32):
        ok = torch.full((t, heads, d), 7.0, dtype=out_type, device="cuda")
        ov = ok.clone()
        lc.ar_kv4_read(h, slots.cuda(), data, scales, ok, ov)
        for got, ref in ((ok, kk), (ov, vv)):
            for i, s in enumerate(slots.tolist()):
                row = ref[s // page, :, s % page] if 0 <= s < pages * page else torch.zeros(heads, d).double()
                assert torch.equal(got[i].cpu().double(), row), (i, s)
    lc.ar_kv4_destroy(h)


def test_every_bfloat16_value_is_quantised_as_the_definition_says(lc):
    """All 65536 bfloat16 values, each beside a largest value that sets the scale: its own, and
    scales at which it falls on every part of the code's range."""
    h = lc.ar_kv4_create(1, 64, 1024)
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = bits.view(BF).view(-1, 16)
    rows = []
    for factor in (1.0, 2.0, 8.0, 64.0):
        top = torch.where(torch.isfinite(x.float()), x.float().abs(), 0.0).amax(-1, keepdim=True) * factor
        pad = top.clamp(max=3.0e38).to(BF).expand(-1, 16)
        rows.append(torch.cat([x, pad], dim=1))
    rows = torch.cat(rows).view(-1, 1, 64)
    t = rows.shape[0]
    k, v = rows.cuda(), rows.flip(0).contiguous().cuda()
    data, scales = _empty(lc, h, -(-t // 1024))
    slots = torch.arange(t)
    lc.ar_kv4_append(h, k, v, slots.cuda(), data, scales)
    out = [torch.empty(t, 1, 64, device="cuda") for _ in range(2)]
    lc.ar_kv4_read(h, slots.cuda(), data, scales, *out)
    for got, src in zip(out, (k, v)):
        want = R.dequantise(*R.quantise(src.float().cpu()))
        got = got.cpu().double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        fine = ~torch.isnan(want)
        assert torch.equal(got[fine], want[fine])
    lc.ar_kv4_destroy(h)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t,hq,hkv,d,rot,inter,page", [
    (1, 8, 1, 128, 128, False, 16), (7, 6, 2, 64, 32, True, 32), (19, 3, 3, 96, 96, False, 16),
    (5, 4, 2, 192, 96, False, 64), (70, 16, 2, 256, 256, True, 16), (6, 0, 2, 128, 0, False, 16),
])
def test_fused_form_is_the_two_calls(lc, dtype, t, hq, hkv, d, rot, inter, page):
    """ar_kv4_norm_rope_append against ar_qk_norm_rope and ar_kv4_append, bit for bit, and its codes
    against the definition."""
    g = torch.Generator().manual_seed(d + t)
    q, k, v = (torch.randn(t, n, d, generator=g).to(dtype).cuda() for n in (hq, hkv, hkv))
    pos = torch.randint(0, 64, (t,), generator=g).int()
    slots = torch.randperm(t + 2 * page, generator=g)[:t]
    pages = -(-(t + 2 * page) // page)
    if t > 3:
        pos[1], pos[2], slots[3] = -1, 64, -1
    cs = _cos_sin(64, rot).cuda() if rot else None
    posd = pos.cuda() if rot else None
    wq, wk = ((1 + torch.randn(d, generator=g) / 4).to(dtype).cuda() for _ in range(2))
    h = lc.ar_kv4_create(hkv, d, page)
    one, two = _empty(lc, h, pages), _empty(lc, h, pages)
    q1, q2, k2 = torch.full_like(q, 7.0), torch.full_like(q, 7.0), torch.zeros_like(k)
    lc.ar_kv4_norm_rope_append(h, q, k, v, q1, posd, cs, slots.cuda(), *one, wq, wk, 1e-6, inter)
    lc.ar_qk_norm_rope(q, k, q2, k2, posd, cs, wq, wk, 1e-6, inter)
    skip = torch.where(pos < 0, -1, slots) if rot else slots
    lc.ar_kv4_append(h, k2, v, skip.cuda(), *two)
    assert torch.equal(q1.view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    want = _reference_cache(*_empty(lc, h, pages), k2, v, skip.tolist(), page)
    assert torch.equal(one[0].cpu(), want[0]) and torch.equal(one[1].cpu(), want[1])
    lc.ar_kv4_destroy(h)


def test_rows_beyond_32_bit_offsets(lc):
    """Slots whose bytes lie past 4 GiB of the cache."""
    heads, d, page = 8, 128, 64
    pages = (5 << 30) // (heads * page * d)
    h = lc.ar_kv4_create(heads, d, page)
    data = torch.empty(pages, heads, 2, page * d // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, heads, 2, d // 32, page, dtype=torch.uint8, device="cuda")
    x = torch.randn(4, heads, d, device="cuda").to(BF)
    last = pages * page - 1
    slots = torch.tensor([last, last - 5000, (4 << 30) // (heads * d) + 3, 17], device="cuda")
    out = [torch.empty_like(x) for _ in range(2)]
    lc.ar_kv4_append(h, x, -x, slots, data, scales)
    lc.ar_kv4_read(h, slots, data, scales, *out)
    want = R.dequantise(*R.quantise(x.float().cpu()))
    assert torch.equal(out[0].cpu().double(), want) and torch.equal(out[1].cpu().double(), -want)
    assert torch.equal(data[pages - 1, :, 0].view(heads, page, d // 2)[:, page - 1].cpu(),
                       (lambda c: (c[:, 0::2] | c[:, 1::2] << 4).to(torch.uint8))(R.quantise(x[0].float().cpu())[0]))
    lc.ar_kv4_destroy(h)


def test_graph_replays_follow_their_inputs(lc):
    """The step's calls captured once: every replay gives the eager result for what the buffers
    hold then."""
    t, hq, hkv, d, page = 6, 4, 2, 64, 16
    h = lc.ar_kv4_create(hkv, d, page)
    cache, eager = _empty(lc, h, 9), _empty(lc, h, 9)
    q, k, v = (torch.zeros(t, n, d, dtype=BF, device="cuda") for n in (hq, hkv, hkv))
    qo, qe = torch.zeros_like(q), torch.zeros_like(q)
    cached, kv, new = _i32([0] * t), _i32([0] * t), _i32([1] * t)
    pool, pool_out, free = _i32([0, 9]), _i32([0, 0]), _i32(list(range(9)))
    table, qs, refused = _i32([[-1] * 2] * t), _i32([0] * (t + 1)), _i32([0] * t)
    slots, pos = torch.zeros(t, dtype=torch.int64, device="cuda"), _i32([0] * t)
    cs = _cos_sin(64, d).cuda()

    def step(out, c):
        lc.ar_page_tables(cached, new, pool, free, table, kv, qs, slots, pos, pool_out, refused, page)
        lc.ar_kv4_norm_rope_append(h, q, k, v, out, pos, cs, slots, *c)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(qo, cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(qo, cache)
    cache[0].fill_(0xA5), cache[1].fill_(0xFF), table.fill_(-1)
    for i in range(4):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda"))
        before = table.clone()
        graph.replay()
        torch.cuda.synchronize()
        table.copy_(before)
        step(qe, eager)
        assert torch.equal(qo, qe) and torch.equal(cache[0], eager[0]) and torch.equal(cache[1], eager[1])
        assert kv.tolist() == [i + 1] * t
        cached.copy_(kv), pool.copy_(pool_out)
    lc.ar_kv4_destroy(h)
