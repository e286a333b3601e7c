"""The row operators at prompts' sizes: groups of lanes that take several heads one after the other, the
next ones' loads under way, and outputs that go past the caches. `heads_a_group` repeats the rule by
which a launch is split, so that a case here says what it reaches. Norm and rotation against the plain
64-bit form within one rounding, the fused form against the two calls bit for bit, the cache's codes
against their definition."""

import os
import re

import pytest
import torch

from tests import decode_ref as R
from tests.test_gpu_decode_rows import BF, F32, _close, _cos_sin, _empty

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lc():
    import latency_collectives_amd as lc

    return lc


def heads_a_group(tokens, rows, d):
    """pick_run() of ar_decode_rows.hip for rows of all tensors together."""
    with open(os.path.join(ROOT, "latency_collectives_amd", "csrc_decode", "ar_decode_rows.hip")) as f:
        few = int(re.search(r"kFewBlocks = (\d+)", f.read())[1])
    lanes = 8 if d <= 64 else 16 if d <= 128 else 32
    blocks, run = -(-tokens * lanes // 256), 8
    while run > 1 and blocks * -(-rows // run) < few:
        run //= 2
    return run


def _projection(t, heads, d, dtype, seed):
    """One token's rows side by side, as strided views; rows of very different size."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, sum(heads) * d, generator=g) * torch.exp2(torch.randint(-9, 9, (t, 1), generator=g).float())
    return [y.view(t, -1, d) for y in x.to(dtype).cuda().split([h * d for h in heads], dim=1)]


def _positions(t, rows, seed):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, rows, (t,), generator=g).int()
    pos[3::101], pos[7::103] = -1, rows  # padding, and past the table
    return pos


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t,hq,hkv,d,rot,inter,run", [
    (3000, 17, 5, 128, 128, False, 8), (3001, 9, 17, 128, 64, True, 8), (5003, 5, 9, 64, 64, False, 4),
    (2501, 9, 1, 256, 256, True, 8), (1203, 12, 4, 96, 48, False, 2), (2111, 9, 8, 192, 0, False, 8),
    (1500, 32, 8, 128, 128, False, 4),
])
def test_norm_rope_of_prompts(lc, dtype, t, hq, hkv, d, rot, inter, run):
    assert heads_a_group(t, hq + hkv, d) == run
    q, k = _projection(t, (hq, hkv), d, dtype, t)
    g = torch.Generator().manual_seed(d)
    wq, wk = ((1 + torch.randn(d, generator=g) / 4).to(dtype) for _ in range(2))
    pos = _positions(t, 300, t) if rot else None
    cs = _cos_sin(300, rot) if rot else None
    dev = [None if x is None else x.cuda() for x in (pos, cs, wq, wk)]
    q_out = torch.full((t, hq + 1, d), 7.0, dtype=dtype, device="cuda")
    k_out = torch.full((t, hkv, d), 7.0, dtype=dtype, device="cuda")
    lc.ar_qk_norm_rope(q, k, q_out[:, :hq], k_out, *dev, 1e-5, inter)
    assert (q_out[:, hq] == 7.0).all()
    live = slice(None) if pos is None else pos >= 0
    for got, x, w in ((q_out[:, :hq], q, wq), (k_out, k, wk)):
        want = R.norm_rope(x.cpu(), w, cs, pos, 1e-5, inter)
        _close(got.cpu()[live], want[live], dtype, 64.0)
        assert pos is None or (got.cpu()[~live] == 7.0).all()
    # in place: the rows of padding keep what they held
    q_was, k_was = q.cpu(), k.cpu()
    lc.ar_qk_norm_rope(q, k, q, k, *dev, 1e-5, inter)
    for got, ref, was in ((q, q_out[:, :hq], q_was), (k, k_out, k_was)):
        want = ref.cpu() if pos is None else torch.where((pos >= 0)[:, None, None], ref.cpu(), was)
        assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("dtype,t,hq,hkv,d", [(BF, 4100, 33, 7, 128), (F32, 2100, 27, 5, 128), (BF, 9001, 17, 13, 64),
                                              (F32, 3000, 9, 3, 256)])
def test_outputs_past_the_caches(lc, dtype, t, hq, hkv, d):
    """More than 32 MiB of whole lines, and the same rows through the caches in smaller calls."""
    assert t * (hq + hkv) * d * (2 if dtype == BF else 4) > 32 << 20
    assert heads_a_group(t, hq + hkv, d) == 8
    q, k = _projection(t, (hq, hkv), d, dtype, t)
    wq, wk = ((1 + torch.randn(d, device="cuda") / 4).to(dtype) for _ in range(2))
    pos, cs = _positions(t, 300, t), _cos_sin(300, d)
    dev = (pos.cuda(), cs.cuda(), wq, wk)
    q_out, k_out = (torch.full((t, h, d), 7.0, dtype=dtype, device="cuda") for h in (hq, hkv))
    lc.ar_qk_norm_rope(q, k, q_out, k_out, *dev, 1e-6)
    some = torch.arange(0, t, 13)
    some = some[pos[some] >= 0]
    for got, x, w in ((q_out, q, wq), (k_out, k, wk)):
        _close(got[some], R.norm_rope(x[some].cpu(), w.cpu(), cs, pos[some], 1e-6, False), dtype, 64.0)
    q2, k2 = torch.full_like(q_out, 7.0), torch.full_like(k_out, 7.0)
    for a in range(0, t, 97):
        part = slice(a, a + 97)
        lc.ar_qk_norm_rope(q[part], k[part], q2[part], k2[part], dev[0][part], *dev[1:], 1e-6)
    assert torch.equal(q_out.view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(k_out.view(torch.uint8), k2.view(torch.uint8))
    # in place
    q_was, k_was = q.clone(), k.clone()
    lc.ar_qk_norm_rope(q, k, q, k, *dev, 1e-6)
    live = (dev[0] >= 0)[:, None, None]
    assert torch.equal(q.contiguous().view(torch.uint8), torch.where(live, q_out, q_was).view(torch.uint8))
    assert torch.equal(k.contiguous().view(torch.uint8), torch.where(live, k_out, k_was).view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t,hq,hkv,d,rot,inter,page,run", [
    (2500, 9, 9, 128, 128, False, 16, 8), (2501, 17, 5, 128, 64, False, 32, 8), (2503, 5, 9, 128, 128, True, 16, 4),
    (5001, 9, 9, 64, 32, False, 64, 8), (1301, 12, 5, 256, 256, False, 16, 4), (1307, 9, 6, 192, 96, False, 128, 4),
    (1800, 5, 5, 96, 96, False, 16, 2),
])
def test_fused_form_of_prompts(lc, dtype, t, hq, hkv, d, rot, inter, page, run):
    """The fused form against ar_qk_norm_rope and ar_kv4_append, and the codes against the definition:
    rows of one token pass through one place of LDS one after the other."""
    assert heads_a_group(t, hq + 2 * hkv, d) == run
    q, k, v = _projection(t, (hq, hkv, hkv), d, dtype, t)
    pos, cs = _positions(t, 300, t), _cos_sin(300, rot)
    g = torch.Generator().manual_seed(t + 1)
    pages = -(-t // page) + 3
    slots = torch.randperm(pages * page, generator=g)[:t]
    slots[5::97], slots[6::89] = -1, pages * page
    wq, wk = ((1 + torch.randn(d, generator=g) / 4).to(dtype).cuda() for _ in range(2))
    h = lc.ar_kv4_create(hkv, d, page)
    one, two = _empty(lc, h, pages), _empty(lc, h, pages)
    q1, q2 = (torch.full((t, hq, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    k2 = torch.zeros(t, hkv, d, dtype=dtype, device="cuda")
    lc.ar_kv4_norm_rope_append(h, q, k, v, q1, pos.cuda(), cs.cuda(), slots.cuda(), *one, wq, wk, 1e-6, inter)
    lc.ar_qk_norm_rope(q, k, q2, k2, pos.cuda(), cs.cuda(), wq, wk, 1e-6, inter)
    stored = torch.where(pos < 0, -1, slots)
    lc.ar_kv4_append(h, k2, v, stored.cuda(), *two)
    assert torch.equal(q1.view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    there = (stored >= 0) & (stored < pages * page)
    at = stored[there]
    for got, x in zip(R.unpack(one[0].cpu(), one[1].cpu(), page), (k2, v)):
        want = R.dequantise(*R.quantise(x.float().cpu()[there]))
        rows = got[at // page, :, at % page]
        assert torch.equal(torch.isnan(rows), torch.isnan(want))
        assert torch.equal(rows.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
    # what no token went to stays as it was
    free = torch.ones(pages * page, dtype=torch.bool)
    free[at] = False
    left = one[1].cpu().permute(0, 4, 1, 2, 3).reshape(pages * page, -1)[free]
    assert (left == 0xFF).all()
    lc.ar_kv4_destroy(h)


def test_append_of_many_heads(lc):
    """Keys and values of 17 heads a token into the cache: runs of eight heads and a shorter one."""
    t, heads, d, page = 1700, 17, 128, 32
    assert heads_a_group(t, 2 * heads, d) == 8
    for dtype in (BF, F32):
        k, v = _projection(t, (heads, heads), d, dtype, 11)
        h = lc.ar_kv4_create(heads, d, page)
        pages = -(-t // page)
        data, scales = _empty(lc, h, pages)
        slots = torch.randperm(pages * page)[:t]
        lc.ar_kv4_append(h, k, v, slots.cuda(), data, scales)
        ko, vo = (torch.zeros(t, heads, d, device="cuda") for _ in range(2))
        lc.ar_kv4_read(h, slots.cuda(), data, scales, ko, vo)
        for got, read, x in zip(R.unpack(data.cpu(), scales.cpu(), page), (ko, vo), (k, v)):
            want = R.dequantise(*R.quantise(x.float().cpu()))
            assert torch.equal(got[slots // page, :, slots % page], want)
            assert torch.equal(read.cpu().double(), want)
        lc.ar_kv4_destroy(h)
