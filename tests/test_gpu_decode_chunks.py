"""ar_kv4_attention where requests bring many rows (prompt chunks, mixed batches) on the GPU, against
the plain 64-bit form within the bound of its roundings, as in test_gpu_decode_attention. Tables are
wide, their columns beyond a request's pages out of range: the width is what lets a few short
requests take the tiles of 128 rows.

A bfloat16 query enters the product as two e4m3 values with a scale for 32 elements, the largest of
which is in [2^7, 2^8) of it. Elements down to 2^-6 of the largest arrive exactly. Smaller ones leave
at most 2^-3 to the lower part, which holds that to 2^-5 of itself: off by 2^-8, 2^-15 of the largest;
and the product drops, of each lower part times a key's code, what is below 2^-7 (2^-13 of the largest
of eight products, below 2^10 of a scale 2^-4): 2^-14 of the largest times the key's scale."""

import pytest
import torch

from tests import decode_ref as R
from tests.test_gpu_decode_attention import BF, F32, Case

pytestmark = pytest.mark.gpu


class Chunks(Case):
    """A case whose table is wide enough for the tiles of 128 rows."""

    def __init__(self, lc, reqs, hq, hkv, d, page, dtype, **kw):
        super().__init__(lc, reqs, hq, hkv, d, page, dtype, **kw)
        assert sum(self.new) * (hq // hkv) > 128 * len(reqs)
        n, width = self.table.shape
        wide = torch.full((n, (1 << 21) // page + 5), -1, dtype=torch.int32, device="cuda")
        wide[:, 3::5] = 2 ** 31 - 1
        wide[:, :width] = self.table
        self.table = wide


@pytest.fixture(scope="module")
def lc():
    import latency_collectives_amd as lc

    return lc


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("hq,hkv,page,window", [(4, 2, 16, 0), (3, 3, 32, 0), (12, 2, 64, 0), (8, 1, 16, 50),
                                                (10, 2, 1024, 1), (71, 1, 16, 0)])
def test_chunks(lc, d, hq, hkv, page, window):
    reqs = [(160, 200), (1, 40), (330, 330), (133, 300), (170, 170), (0, 10), (229, 233)]
    Chunks(lc, reqs, hq, hkv, d, page, BF, seed=d + hq).call(window=window).check().done()


@pytest.mark.parametrize("tokens", [9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257])
def test_row_counts_around_the_tiles(lc, tokens):
    """One request; rows below, at and above multiples of 16, 32 and 128, with either kind of tile."""
    for hq, extra in ((4, 0), (5, 77), (17, 5)):
        for kind in (Case, Chunks) if tokens * hq > 128 else (Case,):
            kind(lc, [(tokens, tokens + extra)], hq, 1, 128, 16, BF, seed=tokens).call().check().done()


@pytest.mark.parametrize("window", [0, 1, 31, 32, 33, 700])
def test_long_chunks_in_parts(lc, window):
    """Few tiles over many tokens: every tile is cut over workgroups. A second call finds the
    workspace as the first did and gives the same bits."""
    c = Chunks(lc, [(70, 6000), (3, 10), (1, 5000)], 16, 2, 128, 64, BF).call(window=window).check()
    first, first_lse = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.out.fill_(7.0), c.lse.fill_(7.0)
        c.call(window=window)
        assert torch.equal(c.out, first) and torch.equal(c.lse, first_lse)
    c.done()


def test_prompts_from_nothing(lc):
    """Tiles whose ranges grow from one token to the prompt's length."""
    for d in (64, 128):
        Chunks(lc, [(700, 700), (333, 333), (1, 1), (64, 64)], 4, 2, d, 16, BF).call().check().done()


@pytest.mark.parametrize("window", [0, 5])
def test_rows_that_see_nothing(lc, window):
    reqs = [(140, 20), (50, 0), (33, -5), (40, 39), (200, 300)]
    c = Chunks(lc, reqs, 6, 2, 128, 16, BF).call(window=window).check()
    assert (c.out[:120] == 0).all() and (c.out[140:190] == 0).all()
    c.done()
    c = Chunks(lc, [(150, 0)], 2, 1, 64, 16, BF).call().check()
    assert (c.out == 0).all()
    c.done()


def test_nan_keys_and_values_reach_only_rows_that_see_them(lc):
    for d in (96, 128, 256):
        for which, window in ((0, 0), (1, 0), (1, 8), (0, 8)):
            c = Chunks(lc, [(60, 200), (90, 90), (50, 150)], 4, 2, d, 16, BF)
            pos = 170
            slot = int(c.table[0, pos // 16]) * 16 + pos % 16
            k, v = torch.ones(2, 1, 2, d, device="cuda")
            (k, v)[which][0, 1, 40] = float("nan")
            c.lc.ar_kv4_append(c.h, k, v, torch.tensor([slot], device="cuda"), c.data, c.scales)
            c.call(window=window).check()
            assert torch.isnan(c.out).any() and not torch.isnan(c.out[:, :2]).any()
            assert not torch.isnan(c.out[:30]).any() and not torch.isnan(c.out[60:]).any()
            if which == 1:  # one group of 32 elements
                assert not torch.isnan(c.out[:, :, :32]).any() and not torch.isnan(c.out[:, :, 64:]).any()
            c.done()


def test_extreme_queries_stay_in_their_rows(lc):
    c = Chunks(lc, [(66, 200)], 4, 2, 64, 16, BF)
    clean = c.call().out.clone()
    c.q[1, 0, 3], c.q[2, 1, 0], c.q[3, 3], c.q[40, 2, 63] = float("inf"), float("nan"), 3e38, float("-inf")
    c.call()
    same = torch.ones(66, 4, dtype=torch.bool, device="cuda")
    same[1, 0] = same[2, 1] = same[3, 3] = same[40, 2] = False
    assert torch.equal(c.out[same], clean[same])
    assert torch.isnan(c.out[1, 0]).all() and torch.isnan(c.out[2, 1]).all() and torch.isnan(c.out[40, 2]).all()
    c.done()


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
def test_queries_of_mixed_size(lc, d):
    """Elements 2^-30 to 2^4 of each other in one group, zero rows, subnormal rows."""
    g = torch.Generator().manual_seed(d)
    c = Chunks(lc, [(70, 90)], 4, 2, d, 16, BF)
    q = torch.randn(70, 4, d, generator=g) * torch.exp2(torch.randint(-30, 5, (70, 4, d), generator=g).float())
    q[3], q[5] = 0.0, torch.randn(4, d, generator=g) * 2.0 ** -130
    c.q = q.to(BF).cuda()
    c.call()
    out, lse, bound, lse_bound = c.want()
    k, v = R.unpack(c.data.cpu(), c.scales.cpu(), 16)
    ids = c.table[0].long().cpu()[:6]
    k, v = (x[ids].transpose(0, 1).reshape(2, -1, d)[:, :90] for x in (k, v))
    qq = c.q.cpu().double()
    # what scores are off by; twice that moves a probability
    most = qq.abs().unflatten(-1, (-1, 32)).amax(-1)  # [70, 4, d / 32]
    steps = torch.exp2(c.scales[:, :, 0].cpu()[ids].double() - 127).permute(1, 0, 3, 2).reshape(2, -1, d // 32)[:, :90]
    size = 2.0 ** -15 * k.abs().unflatten(-1, (-1, 32)).sum(-1) + 2.0 ** -14 * 32 * steps  # [2, 90, d / 32]
    off = c.scale * torch.stack([(most[:, h] @ size[h // 2].T).amax(-1) for h in range(4)], dim=1)
    bound = bound + 2 * off[..., None] * v.abs().amax()
    assert ((c.out.cpu().double() - out).abs() <= bound).all()
    assert ((c.lse.cpu().double() - lse).abs() <= lse_bound + off).all()
    c.done()


@pytest.mark.parametrize("scale,sharp", [(1.0, 3.0), (0.0, 1.0), (-0.5, 1.0), (30.0, 2.0), (1e-30, 1.0)])
def test_scales_and_sharp_rows(lc, scale, sharp):
    Chunks(lc, [(64, 900), (90, 333)], 4, 2, 128, 16, BF, sharp=sharp).call(scale=scale).check().done()


def test_bad_pages_count_as_masked(lc):
    c = Chunks(lc, [(50, 200), (64, 64), (40, 90)], 4, 1, 128, 16, BF)
    c.table[0, 2], c.table[1, 0], c.table[1, 3], c.table[0, 9] = -1, 1 << 30, c.data.shape[0], -7
    c.kv_len[2] = c.kv[2] = 3000
    c.call().check().done()
    c = Chunks(lc, [(80, 80)], 2, 1, 64, 16, BF)
    c.table.fill_(-3)
    c.call().check()
    assert (c.out == 0).all()
    c.done()


def test_strided_queries_and_outputs_and_no_lse(lc):
    c = Chunks(lc, [(37, 77), (81, 500), (20, 20)], 6, 2, 64, 32, BF).call().check()
    t = c.q.shape[0]
    wide = torch.zeros(t, 10, 64, dtype=BF, device="cuda")
    wide[:, 2:8] = c.q
    by_head = torch.full((6, t + 1, 64), 7.0, dtype=BF, device="cuda")
    out = by_head[:, :t].transpose(0, 1)
    lc.ar_kv4_attention(c.h, wide[:, 2:8], c.data, c.scales, c.table, c.kv_len, c.q_start, out)
    assert torch.equal(out, c.out) and (by_head[:, t] == 7.0).all()
    c.done()


def test_starts_that_overlap_or_leave_gaps(lc):
    """Rows that no request covers stay; starts out of order touch nothing outside the tensors, and
    the next call is as any other."""
    c = Chunks(lc, [(60, 80), (70, 90)], 4, 2, 128, 16, BF).call().check()
    want, want_lse = c.out.clone(), c.lse.clone()
    for starts in ([130, -7, 999], [0, 130, 0], [130, 0, 130]):
        bad = torch.tensor(starts, dtype=torch.int32, device="cuda")
        lc.ar_kv4_attention(c.h, c.q, c.data, c.scales, c.table, c.kv_len, bad, c.out, c.lse)
    c.out.fill_(7.0), c.lse.fill_(7.0)
    c.call()
    assert torch.equal(c.out, want) and torch.equal(c.lse, want_lse)
    q = torch.cat([c.q, c.q])
    out = torch.full_like(q, 7.0)
    lc.ar_kv4_attention(c.h, q, c.data, c.scales, c.table, c.kv_len, c.q_start, out)
    assert torch.equal(out[:130], c.out) and (out[130:] == 7.0).all()
    c.done()


def test_many_ragged_requests(lc):
    """More requests than a wave has lanes, most with one token, a few with long chunks."""
    g = torch.Generator().manual_seed(4)
    reqs = []
    for i in range(150):
        m = 1 if i % 7 else int(torch.randint(60, 200, (1,), generator=g))  # 20 tokens on average
        reqs.append((m, m + int(torch.randint(0, 300, (1,), generator=g))))
    Chunks(lc, reqs, 16, 2, 64, 16, BF).call().check().done()


def test_both_kinds_of_tiles_agree(lc):
    """The same request with either kind: each within the bound of the same values."""
    for kind in (Case, Chunks):
        kind(lc, [(64, 3000)], 8, 1, 128, 16, BF, seed=7).call().check().done()


def test_another_stream_and_graph_replays(lc):
    c = Chunks(lc, [(64, 3000), (33, 50), (41, 77)], 8, 1, 128, 16, BF)
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
    for lens in ([3000, 50, 77], [65, 17, 2], [2048, 0, 64], [3000, 50, 77]):
        c.kv_len.copy_(torch.tensor(lens)), c.q.copy_(torch.randn(c.q.shape))
        c.kv = lens
        graph.replay()
        torch.cuda.synchronize()
        c.call().check()
        assert torch.equal(out, c.out) and torch.equal(lse, c.lse)
    c.done()


def test_binary32_chunks(lc):
    """Binary32 stays with the small tiles whatever the rows."""
    Chunks(lc, [(130, 400), (1, 7), (64, 64)], 6, 2, 128, 32, F32).call().check().done()
