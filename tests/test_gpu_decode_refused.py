"""latency_collectives_amd.decode_step where requests are refused or a step is padded: their tokens come
back as they were, whatever earlier steps left in the buffers, and refusals are kept."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ranks", [1, 2])
def test_tokens_without_a_place_come_back_as_they_were(ranks):
    from latency_collectives_amd.decode_step import DecodeStep

    hidden = 256
    run = DecodeStep(ranks, 2, 3, 64, 60, q_heads=8, kv_heads=2, head_dim=64, hidden=hidden, page=16, seed=3)
    run.pool[0][1] = 4  # pages: the first request's three and one more
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def step(new, tokens, dirt):
        for buf in run.q_out + run.attended:
            buf.fill_(dirt)
        x = torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16()
        return x, run(x, torch.tensor(new, dtype=torch.int32, device="cuda"))

    # the second request wants two pages of the one that is left; two tokens of padding
    for dirt in (1.0, float("nan")):
        x, xs = step([40, 17, 0], 59, dirt)
        assert run.refused.tolist() == ([0, 1, 0] if dirt == 1.0 else [1, 1, 0])
        lost = slice(40, 59) if dirt == 1.0 else slice(0, 59)
        for y in xs:
            assert torch.equal(y[lost], x[lost])
            assert torch.isfinite(y.float()).all() and torch.equal(y, xs[0])
        if dirt == 1.0:
            assert (xs[0][:40] != x[:40]).any(dim=1).all()
        assert run.refusals.tolist() == run.refused.tolist()
    # all have their place now: refusals of earlier steps are still known
    x, xs = step([1, 3, 0], 4, float("nan"))
    assert run.refused.tolist() == [0, 0, 0] and run.refusals.tolist() == [1, 1, 0]
    assert run.lengths.tolist() == [41, 3, 0]
    for y in xs:
        assert torch.isfinite(y.float()).all() and (y != x).any(dim=1).all()
    run.close()


def test_a_step_past_the_buffers_changes_nothing():
    from latency_collectives_amd.decode_step import DecodeStep

    run = DecodeStep(1, 1, 2, 64, 20, q_heads=4, kv_heads=2, head_dim=64, hidden=128, page=16)
    x = torch.zeros(21, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="20"):
        run(x, torch.tensor([15, 6], dtype=torch.int32, device="cuda"))
    assert run.lengths.tolist() == [0, 0] and run.turn == 0
    run(x[:20], torch.tensor([15, 5], dtype=torch.int32, device="cuda"))
    assert run.lengths.tolist() == [15, 5]
    run.close()
