"""The forms that the attention over packed prompts and over the 8-bit cache takes for many rows, each reached by
its sizes: against the plain 64-bit form (serving_ref.dense_attention, on the GPU), within the bound that its
roundings give."""

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


def compare(got, got_lse, want):
    out, lse, bound, lse_bound = want
    wild = ~torch.isfinite(out)
    assert torch.equal(~torch.isfinite(got), wild), "infinite or NaN in other places"
    assert torch.equal(got[wild & ~out.isnan()], out[wild & ~out.isnan()].to(got.dtype))
    over = ((got.double() - out).abs() - bound)[~wild]
    assert float(over.max()) <= 0, float(over.max())
    assert torch.equal(got_lse.isnan(), lse.isnan())
    live = torch.isfinite(lse)
    over = ((got_lse.double() - lse).abs() - lse_bound)[live]
    assert float(over.max()) <= 0, float(over.max())


def prompts(lc, lens, hq, hkv, d, dtype, window, poke):
    g = torch.Generator(device="cuda").manual_seed(d + window)
    t = sum(lens)
    q, k, v = (torch.randn(t, n, d, generator=g, device="cuda").to(dtype) for n in (hq, hkv, hkv))
    for x, token, head, element, value in poke:
        (k if x == "k" else v)[token, head, element] = value
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    out, lse = torch.full_like(q, 7.0), torch.full((t, hq), 7.0, device="cuda")
    h = lc.ar_prompt_create(hkv, d)
    lc.ar_prompt_attention(h, q, k, v, torch.tensor(starts, dtype=torch.int32, device="cuda"), out, lse, None, window)
    torch.cuda.synchronize()
    lc.ar_prompt_destroy(h)
    for a, b in zip(starts, starts[1:]):
        compare(out[a:b], lse[a:b], S.dense_attention(q[a:b], k[a:b], v[a:b], 1 / math.sqrt(d), window))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("window", [0, 50])
def test_prompts_of_many_rows(lc, dtype, d, window):
    """64 query heads a kv head: more rows than few, tiles of 64 to 192."""
    prompts(lc, [200, 1, 77, 130], 512, 8, d, dtype, window, [])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("window", [0, 50])
def test_prompts_of_many_rows_with_values_that_are_not_finite(lc, dtype, d, window):
    poke = [("v", 33, 0, d - 1, math.nan), ("v", 34, 0, 3, math.inf), ("v", 150, 2, 0, -math.inf), ("v", 199, 7, 17, math.nan),
            ("v", 201, 3, 40, math.inf), ("v", 277, 3, 40, -math.inf), ("v", 300, 3, 40, math.inf), ("k", 290, 5, 9, math.nan)]
    prompts(lc, [200, 1, 77, 130], 512, 8, d, dtype, window, poke)


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("window,bad", [(0, False), (0, True), (200, True)])
def test_prompts_of_large_tiles(lc, d, window, bad):
    """128 query heads a kv head and 600 tokens: tiles of 256 and 384 rows where there are such."""
    poke = [("v", 33, 0, d - 1, math.nan), ("v", 599, 1, 3, math.inf), ("v", 800, 2, 0, -math.inf), ("k", 700, 5, 9, math.nan)]
    prompts(lc, [600, 600], 1024, 8, d, BF, window, poke if bad else [])


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("window,bad", [(0, False), (0, True), (70, True)])
def test_chunks_that_see_few_tokens(lc, d, page, window, bad):
    """64 query heads a kv head over the 8-bit cache, up to 520 tokens: tiles of many rows, the smaller ones where there are two."""
    hq, hkv, reqs = 512, 8, [(130, 520), (131, 400), (1, 1)]
    g = torch.Generator(device="cuda").manual_seed(d + page)
    width = -(-520 // page)
    pages = len(reqs) * width + 3
    h = lc.ar_kv8_create(hkv, d, page)
    data, scales = lc.ar_kv8_cache(h, pages)
    data.copy_(torch.randint(0, 0x7F, data.shape, generator=g, device="cuda", dtype=torch.uint8))
    data |= torch.randint(0, 2, data.shape, generator=g, device="cuda", dtype=torch.uint8) << 7
    data[data == 0xFF] = 0
    scales.copy_(torch.randint(118, 122, scales.shape, generator=g, device="cuda", dtype=torch.uint8))
    table = torch.randperm(pages, generator=g, device="cuda").int()[:len(reqs) * width].view(len(reqs), width)
    if bad:  # NaN codes, seen by some rows of their tiles: a value's, a key's
        for request, token, head, which, element in ((0, 450, 0, 1, 5), (1, 399, 7, 1, d - 1), (1, 300, 3, 0, 9), (0, 519, 2, 1, 0)):
            pg, off = int(table[request, token // page]), token % page
            if which == 0:
                data[pg, head, 0].view(page, d)[off, element] = 0x7F
            else:
                data[pg, head, 1].view(page // 4, d, 4)[off // 4, element, off % 4] = 0xFF
    t = sum(m for m, _ in reqs)
    q = torch.randn(t, hq, d, generator=g, device="cuda").bfloat16()
    out, lse = torch.full_like(q, 7.0), torch.full((t, hq), 7.0, device="cuda")
    starts = [0, 130, 261, 262]
    i32 = dict(dtype=torch.int32, device="cuda")
    lc.ar_kv8_attention(h, q, data, scales, table, torch.tensor([n for _, n in reqs], **i32), torch.tensor(starts, **i32), out, lse,
                        0.02, window)
    torch.cuda.synchronize()
    lc.ar_kv8_destroy(h)
    values = S.unpack(data.cpu(), scales.cpu(), d)[0].cuda()  # [pages, heads, 2, page, d]
    for b, (m, n) in enumerate(reqs):
        kv = values[table[b].long()].permute(2, 0, 3, 1, 4).reshape(2, width * page, hkv, d)[:, :n]
        a = starts[b]
        compare(out[a:a + m], lse[a:a + m], S.dense_attention(q[a:a + m], kv[0], kv[1], 0.02, window))
