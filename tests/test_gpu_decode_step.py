"""latency_collectives_amd.decode_step: the operators together, over prompts and decode steps, on
emulated ranks. Tables and lengths against the plain forms, the attention of every rank's last layer
against the 64-bit form of what its cache holds, the sum of the partial results on every rank."""

import pytest
import torch

from tests import decode_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ranks,page", [(1, 16), (2, 32)])
def test_prompts_and_steps(ranks, page):
    from latency_collectives_amd.decode_step import DecodeStep

    prompts, hidden = [40, 3, 17], 256
    run = DecodeStep(ranks, 2, 3, 64, 80, q_heads=8, kv_heads=2, head_dim=64, hidden=hidden, page=page, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    cached, pool, table = [0, 0, 0], [0, 3 * (64 // page)], run.table.tolist()
    free = run.free.tolist()
    for step, new in enumerate([prompts, [1, 1, 1], [1, 1, 1], [2, 0, 5], [1, 1, 1]]):
        t = sum(new)
        x = torch.randn(t, hidden, device="cuda", generator=g).bfloat16()
        xs = run(x, torch.tensor(new, dtype=torch.int32, device="cuda"))
        want = R.page_tables(cached, new, pool, free, table, t, page)
        table, cached, pool = want[0], want[1], want[5]
        assert run.table.tolist() == table and run.lengths.tolist() == cached
        assert run.slots[:t].tolist() == want[3] and run.positions[:t].tolist() == want[4]
        assert run.refused.tolist() == [0, 0, 0]
        for r in range(ranks):
            data, scales = (c.cpu() for c in run.cache[-1][r])
            k, v = R.unpack(data, scales, page)
            out, _, bound, _ = R.attention(run.q_out[r][:t].cpu(), k, v, run.table.cpu(), cached, want[2], page,
                                           64 ** -0.5, 0)
            assert ((run.attended[r][:t].cpu().double() - out).abs() <= bound).all(), (step, r)
            assert torch.equal(xs[r], xs[0]) and torch.isfinite(xs[r].float()).all()
    run.close()


def test_the_command_runs(capsys):
    from latency_collectives_amd import decode_step

    decode_step.main(["--ranks", "2", "--layers", "1", "--requests", "5", "--prompt", "70", "--steps", "3"])
    assert "us a decode step" in capsys.readouterr().out
