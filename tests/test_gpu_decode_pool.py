"""ar_page_tables with a free list whose first entry lies before it: no page is given twice."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("first", [-1, -3, -2 ** 31])
def test_a_pool_that_begins_before_its_list(first):
    import latency_collectives_amd as lc

    free, page = _i32([10, 11, 12, 13, 14]), 16
    kv, pool = [_i32([0, 0]), _i32([0, 0])], [_i32([first, 5]), _i32([0, 0])]
    table = _i32([[-1] * 3] * 2)
    given = []
    for step in range(3):
        a, b = step % 2, 1 - step % 2
        slots, pos = torch.zeros(40, dtype=torch.int64, device="cuda"), _i32([0] * 40)
        q, refused = _i32([0] * 3), _i32([0] * 2)
        lc.ar_page_tables(kv[a], _i32([16, 16]), pool[a], free, table, kv[b], q, slots, pos, pool[b], refused, page)
        given += [p for p in table[:, step].tolist() if p >= 0]
        assert pool[b].tolist() == [len(given), 5]
        assert refused.tolist() == ([0, 0] if step < 2 else [0, 1])
    assert given == [10, 11, 12, 13, 14]
