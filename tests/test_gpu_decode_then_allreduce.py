"""The AllReduce in a process whose other queues have been used, as a serving program's are: work on a
second stream and replayed graphs moves the XCD that a queue's first workgroup goes to, also between a
handle's making and its calls. Results match the oracle as in a process of one queue."""

import numpy as np
import pytest
import torch

from latency_collectives_amd import inputs as I
from tests import gpu_util as U
from tests.test_gpu_decode_attention import BF, Case

pytestmark = pytest.mark.gpu


def _use_other_queues(times):
    import latency_collectives_amd as lc

    c = Case(lc, [(1, 500), (2, 77)], 8, 2, 64, 16, BF)
    for _ in range(times):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.call()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.call()
        graph.replay()
        torch.cuda.synchronize()
    c.check().done()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "i32"])
@pytest.mark.parametrize("n", [2, 4, 8, 16])
def test_allreduce_after_other_queues(n, dtype):
    counts = (4, 1000, 65536, 300001)
    with U.handle(n, counts[-1] * I.ELEM_BYTES[dtype], dtype) as h:
        for round_ in range(3):
            for i, count in enumerate(counts):
                dist = "int20" if dtype == "i32" else "normal"
                x = np.ascontiguousarray(I.rank_inputs(dist, dtype, n, count, workload=0, size_idx=i,
                                                       iteration=round_))
                for algo in U.ALGO_NAMES:
                    U.assert_matches(U.run_allreduce(h, x, algo), x, algo, dtype)
            _use_other_queues(round_ + 1)
