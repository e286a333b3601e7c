"""latency_collectives_amd.decode_step over the 8-bit cache, with packed prompts, copies that share pages,
requests given back and compactions: tables, lengths and the free list against the plain forms, the attention
of every rank's last layer against the 64-bit form of what its cache holds."""

import pytest
import torch

from tests import decode_ref as R
from tests import serving_ref as S

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Run:
    """A DecodeStep beside lists."""

    def __init__(self, ranks, bits, page, requests, pages=None):
        from latency_collectives_amd.decode_step import DecodeStep

        self.bits, self.page, self.ranks = bits, page, ranks
        self.run = DecodeStep(ranks, 2, requests, 96, 120, q_heads=8, kv_heads=2, head_dim=64, hidden=256, page=page,
                              seed=3, bits=bits)
        self.kv, self.pool = [0] * requests, [0, self.run.free.numel()]
        self.table, self.free = self.run.table.tolist(), self.run.free.tolist()
        self.shares = [0] * len(self.free)
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(5)

    def step(self, new, fresh=False):
        t = sum(new)
        x = torch.randn(t, 256, device="cuda", generator=self.g).bfloat16()
        xs = self.run(x, i32(new), fresh=fresh)
        want = R.page_tables(self.kv, new, self.pool, self.free, self.table, t, self.page)
        self.table, self.kv, self.pool = want[0], want[1], want[5]
        self.check()
        for r in range(self.ranks):
            q, got = self.run.q_out[r][:t].cpu(), self.run.attended[r][:t].cpu().double()
            assert torch.equal(xs[r], xs[0]) and torch.isfinite(xs[r].float()).all()
            if fresh:
                continue
            data, scales = (c.cpu() for c in self.run.cache[-1][r])
            if self.bits == 8:
                x8, _ = S.unpack(data, scales, 64)
                k, v = x8[:, :, 0], x8[:, :, 1]
            else:
                k, v = R.unpack(data, scales, self.page)
            out, _, bound, _ = R.attention(q, k, v, self.run.table.cpu(), self.kv, want[2], self.page, 64 ** -0.5, 0)
            assert ((got - out).abs() <= bound).all(), r
        return xs[0]

    def fork(self, src, dst):
        refused = self.run.fork(i32(src), i32(dst))
        self.table, self.shares, self.kv, self.pool, _, _, want = S.fork(src, dst, self.kv, self.table, self.shares,
                                                                         self.pool, self.free, self.page)
        assert refused.tolist() == want
        self.check()

    def release(self, requests):
        self.run.release(i32(requests))
        self.shares, self.free, self.kv, self.pool = S.free_pages(requests, self.kv, self.table, self.shares, self.pool,
                                                                  self.free, self.page)
        self.check()

    def compact(self):
        self.run.compact()
        self.table, self.shares, self.pool, _, _ = S.compact(self.kv, self.table, self.shares, self.page, len(self.free))
        self.free = list(range(len(self.free)))
        self.check()

    def check(self):
        run = self.run
        assert run.table.tolist() == self.table and run.lengths.tolist() == self.kv
        assert run.pool[run.turn].tolist() == self.pool and run.free.tolist() == self.free
        assert run.shares.tolist() == self.shares


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("ranks,page", [(1, 16), (2, 32)])
def test_lives_of_requests(ranks, bits, page):
    r = Run(ranks, bits, page, 7)
    r.step([40, 3, 17, 0, 0, 0, 0], fresh=True)
    r.step([1, 1, 1, 0, 0, 0, 0])
    r.fork([0, 0, 2, 9], [3, 4, 5, 6])
    r.step([1, 0, 1, 1, 2, 1, 0])  # copies go on by themselves, their shared pages unchanged
    r.release([0, 2, 2])
    r.step([0, 1, 0, 1, 1, 1, 0])
    r.compact()
    r.step([0, 1, 0, 1, 1, 9, 0])
    r.step([33, 0, 5, 0, 0, 0, 8], fresh=True)  # freed rows and pages serve again
    r.fork([3, 0], [0, 6])  # into rows that are taken
    r.compact()
    r.step([1, 1, 1, 1, 1, 1, 1])
    r.release(list(range(7)))
    assert r.pool == [0, len(r.free)] and not any(r.shares)
    r.run.close()


@pytest.mark.parametrize("bits", [4, 8])
def test_a_copy_goes_on_as_its_source_would(bits):
    """A request and its copy give the same results for the same tokens."""
    r = Run(1, bits, 16, 2)
    r.step([37, 0])
    r.fork([0], [1])
    for _ in range(20):
        x = torch.randn(1, 256, device="cuda", generator=r.g).bfloat16()
        (y,) = r.run(torch.cat([x, x]), i32([1, 1]))
        assert torch.equal(y[0], y[1])
    r.run.close()


def test_packed_prompts_against_the_definition():
    """Prompts that attend over their own keys and values, as the projection gave them."""
    from latency_collectives_amd import decode_step

    r = Run(2, 8, 16, 3)
    new = [50, 1, 33]
    x = torch.randn(84, 256, device="cuda", generator=r.g).bfloat16()
    calls = []
    inner = decode_step.lc.ar_prompt_attention

    def spy(h, q, k, v, q_start, out):
        inner(h, q, k, v, q_start, out)
        calls.append([t.cpu() for t in (q, k, v, q_start, out)])

    decode_step.lc.ar_prompt_attention = spy
    try:
        r.run(x, i32(new), fresh=True)
    finally:
        decode_step.lc.ar_prompt_attention = inner
    assert len(calls) == 4
    for q, k, v, q_start, got in calls:
        out, _, bound, _ = S.prompt_attention(q, k, v, q_start.tolist(), 64 ** -0.5, 0)
        assert ((got.double() - out).abs() <= bound).all()
    r.run.close()


@pytest.mark.parametrize("extra", [["--bits", "8"], ["--samples", "3"], ["--bits", "8", "--samples", "2", "--packed"]])
def test_the_command_runs(capsys, extra):
    from latency_collectives_amd import decode_step

    decode_step.main(["--ranks", "2", "--layers", "1", "--requests", "5", "--prompt", "70", "--steps", "3", *extra])
    assert "us a decode step" in capsys.readouterr().out
