"""ar_prompt_attention on the GPU against the plain 64-bit form, within the bound that its roundings give
(decode_ref.attention over each request's own tokens)."""

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


class Case:
    def __init__(self, lc, lens, hq, hkv, d, dtype, seed=0, sharp=1.0, pad=0):
        g = torch.Generator().manual_seed(seed)
        self.lc, self.d = lc, d
        self.h = lc.ar_prompt_create(hkv, d)
        t = sum(lens) + pad
        qkv = torch.randn(t, (hq + 2 * hkv) * d, generator=g)
        qkv[:, :hq * d] *= sharp
        qkv = qkv.to(dtype).cuda()
        self.q, self.k, self.v = (x.view(t, n, d) for x, n in zip(qkv.split([hq * d, hkv * d, hkv * d], dim=1), (hq, hkv, hkv)))
        starts = [0]
        for n in lens:
            starts.append(starts[-1] + n)
        self.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.out = torch.full((t, hq, d), 7.0, dtype=dtype, device="cuda")
        self.lse = torch.full((t, hq), 7.0, device="cuda")

    def call(self, scale=None, window=0):
        self.scale, self.window = 1 / math.sqrt(self.d) if scale is None else scale, window
        self.lc.ar_prompt_attention(self.h, self.q, self.k, self.v, self.q_start, self.out, self.lse, scale, window)
        return self

    def check(self):
        out, lse, bound, lse_bound = S.prompt_attention(self.q.cpu(), self.k.cpu(), self.v.cpu(), self.q_start.tolist(),
                                                        self.scale, self.window)
        got, got_lse = self.out.cpu().double(), self.lse.cpu().double()
        free = torch.ones(out.shape[0], dtype=torch.bool)
        at = self.q_start.clamp(0, out.shape[0]).tolist()
        for a, b in zip(at, at[1:]):
            free[a:b] = False
        assert (got[free] == 7).all() and (got_lse[free] == 7).all()  # nobody's tokens keep their rows
        got, got_lse, out, lse, bound, lse_bound = (x[~free] for x in (got, got_lse, out, lse, bound, lse_bound))
        wild = ~torch.isfinite(out)
        assert torch.equal(~torch.isfinite(got), wild), "infinite or NaN in other places"
        over = ((got - out).abs() - bound)[~wild]
        assert over.numel() == 0 or float(over.max()) <= 0, float(over.max())
        assert torch.equal(torch.isnan(got_lse), torch.isnan(lse))
        live = torch.isfinite(lse)
        over = ((got_lse - lse).abs() - lse_bound)[live]
        assert over.numel() == 0 or float(over.max()) <= 0, float(over.max())
        return self

    def done(self):
        torch.cuda.synchronize()
        self.lc.ar_prompt_destroy(self.h)


LENS = [1, 2, 15, 16, 17, 31, 32, 33, 0, 63, 65, 127, 129, 0, 200]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (6, 2), (7, 7), (34, 2), (130, 1)])
def test_ragged_prompts(lc, dtype, d, hq, hkv):
    Case(lc, LENS, hq, hkv, d, dtype, seed=d + hq).call().check().done()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 2 ** 31 - 1])
def test_windows(lc, dtype, d, window):
    Case(lc, LENS + [400], 4, 2, d, dtype, seed=window % 1000).call(window=window).check().done()


@pytest.mark.parametrize("dtype,n", [(BF, 5003), (F32, 1501), (BF, 1)])
@pytest.mark.parametrize("window", [0, 700])
def test_a_long_prompt_in_parts(lc, dtype, n, window):
    """One request over the whole device; the same bits at every call."""
    c = Case(lc, [n], 2, 1, 128, dtype).call(window=window).check()
    first, first_lse = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.out.fill_(7.0), c.lse.fill_(7.0)
        c.call(window=window)
        assert torch.equal(c.out, first) and torch.equal(c.lse, first_lse)
    c.done()


@pytest.mark.parametrize("scale,sharp", [(1.0, 3.0), (0.0, 1.0), (-0.5, 1.0), (30.0, 2.0)])
def test_scales_and_sharp_rows(lc, scale, sharp):
    for dtype in (BF, F32):
        Case(lc, [333, 40], 4, 2, 64, dtype, sharp=sharp).call(scale=scale).check().done()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(lc, dtype, d, bad):
    for window in (0, 8, 50):
        c = Case(lc, [150, 60, 70], 6, 2, d, dtype, seed=window)
        for token, head, element in ((33, 0, d - 1), (149, 1, 0), (150, 0, 17), (209, 1, 40), (279, 0, 3)):
            c.v[token, head, element] = bad
        c.call(window=window).check()
        assert (~torch.isfinite(c.out)).any() and torch.isfinite(c.out).any() and torch.isfinite(c.lse).all()
        c.done()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_keys_that_are_not_finite(lc, dtype):
    """NaN keys make NaN the rows that see them; masked ones, those of other requests too, nothing."""
    for window in (0, 20):
        c = Case(lc, [100, 130], 4, 1, 128, dtype)
        c.k[60, 0, 5] = math.nan
        c.k[229, 0, 7] = math.nan
        c.call(window=window).check()
        assert torch.isnan(c.out[60]).all() and not torch.isnan(c.out[:60]).any() and not torch.isnan(c.out[100:229]).any()
        c.done()


def test_starts_that_are_out_of_order_or_range(lc):
    """Starts are taken between 0 and ntokens, an end before its start is an empty request, and what no
    request covers stays."""
    for starts in ([0, 40, 30, 90], [-5, 20, 2 ** 31 - 1], [10, 60], [100, 100, 100], [2 ** 31 - 1, -2 ** 31]):
        c = Case(lc, [100], 4, 2, 64, BF)
        c.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        if starts == [0, 40, 30, 90]:  # tokens 30 to 40 are in two requests: whoever writes last
            c.call()
            torch.cuda.synchronize()
            assert torch.isfinite(c.out.float()).all() and (c.out[90:] == 7).all()
        else:
            c.call().check()
        c.done()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_other_layouts(lc, dtype):
    """Heads before tokens, padded rows, broadcast keys."""
    c = Case(lc, [70, 9], 6, 2, 96, dtype)
    c.call().check()
    first = c.out.clone()
    q, k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (c.q, c.k, c.v))
    out = torch.full((79, 6, 120), 5.0, dtype=dtype, device="cuda")
    c.lc.ar_prompt_attention(c.h, q, k, v, c.q_start, out[..., 16:112])
    assert torch.equal(out[..., 16:112], first) and (out[..., :16] == 5).all() and (out[..., 112:] == 5).all()
    c.k = c.k[:1].expand(79, 2, 96)
    c.v = c.v[:, :1].expand(79, 2, 96)
    c.call().check().done()


def test_padding_after_the_last_prompt(lc):
    for dtype in (BF, F32):
        c = Case(lc, [40, 3], 4, 2, 128, dtype, pad=11)
        c.k[43:], c.v[43:], c.q[43:] = math.nan, math.inf, math.nan
        c.call().check().done()


def test_two_handles_on_two_streams_and_a_graph(lc):
    a, b = Case(lc, [900, 3], 8, 1, 128, BF, seed=1), Case(lc, [50, 700], 8, 1, 128, BF, seed=2)
    want = []
    for c in (a, b):
        c.call().check()
        want.append(c.out.clone())
        c.out.fill_(7.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, c in zip(streams, (a, b)):
        with torch.cuda.stream(s):
            for _ in range(5):
                c.call()
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        a.call()
    for starts in ([0, 900, 903], [0, 450, 700], [5, 5, 903], [0, 900, 903]):
        a.q_start.copy_(torch.tensor(starts, dtype=torch.int32))
        a.q.normal_()
        torch.cuda.synchronize()
        a.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = a.out.clone()
        a.out.fill_(7.0)
        a.call()
        assert torch.equal(a.out, got)
        a.lse.copy_(torch.where((a.out[..., 0] == 7), 7.0, a.lse))
    a.check()
    a.done()
    b.done()


def test_tensors_that_want_gradients_are_refused(lc):
    c = Case(lc, [4], 2, 1, 64, BF)
    with pytest.raises(ValueError, match="gradient"):
        lc.ar_prompt_attention(c.h, c.q.requires_grad_(), c.k, c.v, c.q_start, c.out)
    c.done()
