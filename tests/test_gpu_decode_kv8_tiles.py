"""ar_kv8_attention with requests of several dozen to several hundred rows, where the call chooses between tiles of 16, 32
and more rows by what each would take: against the plain 64-bit form (serving_ref.dense_attention, on the GPU),
within the bound that its roundings give."""

import math

import pytest
import torch

from tests import serving_ref as S
from tests.test_gpu_decode_attention_forms import compare, lc  # noqa: F401  (lc is the fixture)

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


class Batch:
    """Requests of ragged chunks over an 8-bit cache of random codes: `reqs` of `tokens` new ones in the mean."""

    def __init__(self, lc, d, reqs, tokens, room, hkv=8, group=4, page=32, dtype=BF, seed=0):  # noqa: F811
        g = torch.Generator(device="cuda").manual_seed(seed + d)
        self.lc, self.d, self.page, self.hkv, self.group = lc, d, page, hkv, group
        # pairs of few and many
        self.new = [tokens + (-1) ** i * ((i * 37) % tokens) * (i // 2 * 2 + 1 < reqs) for i in range(reqs)]
        self.kv = [m + (i * 61) % max(room - m, 1) for i, m in enumerate(self.new)]
        self.kv[0] = room
        width = -(-room // page)
        pages = reqs * width + 3
        self.h = lc.ar_kv8_create(hkv, d, page)
        self.data, self.scales = lc.ar_kv8_cache(self.h, pages)
        self.data.copy_(torch.randint(0, 0x7F, self.data.shape, generator=g, device="cuda", dtype=torch.uint8))
        self.data |= torch.randint(0, 2, self.data.shape, generator=g, device="cuda", dtype=torch.uint8) << 7
        self.data[self.data == 0xFF] = 0
        self.scales.copy_(torch.randint(118, 122, self.scales.shape, generator=g, device="cuda", dtype=torch.uint8))
        self.table = torch.randperm(pages, generator=g, device="cuda").int()[:reqs * width].view(reqs, width)
        self.starts = [0]
        for m in self.new:
            self.starts.append(self.starts[-1] + m)
        self.q = torch.randn(self.starts[-1], hkv * group, d, generator=g, device="cuda").to(dtype)

    def poke(self, request, token, head, which, element):
        """A NaN code in a request's key or value."""
        pg, off = int(self.table[request, token // self.page]), token % self.page
        if which == 0:
            self.data[pg, head, 0].view(self.page, self.d)[off, element] = 0x7F
        else:
            self.data[pg, head, 1].view(self.page // 4, self.d, 4)[off // 4, element, off % 4] = 0xFF

    def call(self, scale=0.02, window=0):
        i32 = dict(dtype=torch.int32, device="cuda")
        out, lse = torch.full_like(self.q, 7.0), torch.full(self.q.shape[:2], 7.0, device="cuda")
        self.lc.ar_kv8_attention(self.h, self.q, self.data, self.scales, self.table, torch.tensor(self.kv, **i32),
                                 torch.tensor(self.starts, **i32), out, lse, scale, window)
        torch.cuda.synchronize()
        return out, lse

    def check(self, scale=0.02, window=0):
        out, lse = self.call(scale, window)
        values = S.unpack(self.data.cpu(), self.scales.cpu(), self.d)[0].cuda()  # [pages, heads, 2, page, d]
        for b, (m, n) in enumerate(zip(self.new, self.kv)):
            kv = values[self.table[b].long()].permute(2, 0, 3, 1, 4).reshape(2, -1, self.hkv, self.d)[:, :n]
            a = slice(self.starts[b], self.starts[b + 1])
            compare(out[a], lse[a], S.dense_attention(self.q[a], kv[0], kv[1], scale, window))
        return self

    def done(self):
        self.lc.ar_kv8_destroy(self.h)


# Heads of 64, 96, 128, 192 and 256 take tiles of: 32, 32, 32, 192, 192; 32, 128, 128, 192, 192; 256, 384, 384, 192, 192.
SIZES = [(24, 24, 500), (24, 64, 900), (24, 190, 900)]


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("window", [0, 1, 70, 300])
def test_chunks(lc, d, size, window):  # noqa: F811
    Batch(lc, d, *size, page=16 if window == 70 else 64).check(window=window).done()


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("which,window", [(0, 0), (1, 0), (0, 70), (1, 70)])
def test_nan_keys_and_values_reach_only_rows_that_see_them(lc, d, size, which, window):  # noqa: F811
    c = Batch(lc, d, *size, page=16, seed=which)
    for b, head in ((0, 0), (3, 7), (8, 3)):
        for token in (c.kv[b] - 1, c.kv[b] - c.new[b] // 2, (c.kv[b] - c.new[b]) // 2, 0):
            c.poke(b, max(token, 0), head, which, (d - 1, 0, 5)[b % 3])
    c.check(window=window)
    out, _ = c.call(window=window)
    assert torch.isnan(out).any() and not torch.isnan(out).all()
    c.done()


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("size", SIZES)
def test_scales_of_scores(lc, d, size):  # noqa: F811
    c = Batch(lc, d, *size)
    for scale in (-0.02, 0.0, 0.5):
        c.check(scale=scale)
    c.done()


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("size", SIZES)
def test_rows_before_the_first_token_and_pages_that_are_not_there(lc, d, size):  # noqa: F811
    """More new tokens than the length: rows that see nothing are zeros. Ids outside the cache mask their tokens."""
    c = Batch(lc, d, *size)
    c.kv[5], c.kv[6] = c.new[5] // 2, 0
    out, lse = c.call()
    for b in (5, 6):
        none = c.new[b] - c.kv[b]
        a = slice(c.starts[b], c.starts[b] + none)
        assert (out[a] == 0).all() and (lse[a] == -math.inf).all() and torch.isfinite(lse[a.stop:c.starts[b + 1]]).all()
    # the first page of request 2 masked: what its window of the last page sees is as it was
    m = c.new[2]
    before, _ = c.call(window=16)
    keep = c.table.clone()
    c.table[2, 0] = 2 ** 31 - 1
    after, lse = c.call(window=16)
    far = max(0, c.page + 16 - (c.kv[2] - m))  # rows from here on see nothing of the first page
    assert torch.equal(after[c.starts[2] + far:c.starts[3]], before[c.starts[2] + far:c.starts[3]])
    c.table[2] = -1
    out, lse = c.call()
    assert (out[c.starts[2]:c.starts[3]] == 0).all() and (lse[c.starts[2]:c.starts[3]] == -math.inf).all()
    c.table.copy_(keep)
    c.done()


@pytest.mark.parametrize("tokens", [9, 40])
def test_binary32(lc, tokens):  # noqa: F811
    """Tiles of 16 and of 32 rows."""
    for window in (0, 33):
        Batch(lc, 64, 24, tokens, 400, dtype=F32).check(window=window).done()
