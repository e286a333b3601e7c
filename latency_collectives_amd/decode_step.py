"""The attention half of tensor-parallel decoding on emulated ranks, every operator of this package as
a serving program calls it.

    python -m latency_collectives_amd.decode_step [--ranks 4] [--layers 2] [--requests 16] ...

Each rank holds its share of the heads, its slice of the projections and its own 4-bit cache. A step
builds the block tables and slots once, then every layer projects the tokens, normalises and rotates
queries and keys while the new keys and values go into the cache (one launch), attends over the
cache, projects back, and sums the ranks' partial results with the AllReduce. Lengths and the free
list stay on the GPU from step to step. Weights are random: this shows how the calls fit together
and what a step costs, not a model.
"""

from __future__ import annotations

import argparse
import math
import time

import torch

import latency_collectives_amd as lc


class DecodeStep:
    """`ranks` ranks of `layers` attention blocks over a paged cache for up to `requests` requests."""

    def __init__(self, ranks: int, layers: int, requests: int, max_len: int, max_tokens: int,
                 q_heads: int = 32, kv_heads: int = 8, head_dim: int = 128, hidden: int = 2048,
                 page: int = 16, seed: int = 0):
        if kv_heads % ranks or q_heads % kv_heads:
            raise ValueError("kv_heads is a multiple of ranks, q_heads of kv_heads")
        self.ranks, self.layers, self.page, self.dim = ranks, layers, page, head_dim
        self.hq, self.hkv, self.hidden = q_heads // ranks, kv_heads // ranks, hidden
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weights(rows, cols):
            return [[(torch.randn(rows, cols, device="cuda", generator=g) / math.sqrt(rows)).bfloat16()
                     for _ in range(ranks)] for _ in range(layers)]

        self.w_in = weights(hidden, (self.hq + 2 * self.hkv) * head_dim)
        self.w_out = weights(self.hq * head_dim, hidden)
        self.q_norm = torch.ones(head_dim, dtype=torch.bfloat16, device="cuda")
        self.k_norm = torch.ones(head_dim, dtype=torch.bfloat16, device="cuda")
        angle = torch.arange(max_len, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(0, head_dim, 2, dtype=torch.float64, device="cuda") / head_dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], dim=1).float()

        width = -(-max_len // page)
        pages = requests * width
        self.kv = lc.ar_kv4_create(self.hkv, head_dim, page)
        self.cache = [[lc.ar_kv4_cache(self.kv, pages) for _ in range(ranks)] for _ in range(layers)]
        self.sum = lc.ar_create(ranks, max_tokens * hidden * 2, lc.AR_BFLOAT16)

        def i32(*shape):
            return torch.zeros(*shape, dtype=torch.int32, device="cuda")

        # lengths and the pool alternate between two buffers: a step reads one and writes the other
        self.len, self.pool, self.turn = [i32(requests), i32(requests)], [i32(2), i32(2)], 0
        self.pool[0][1] = pages
        self.free = torch.randperm(pages, device="cuda", generator=g).int()
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
        self.refused, self.refusals, self.q_start = i32(requests), i32(requests), i32(requests + 1)
        self.slots = torch.zeros(max_tokens, dtype=torch.int64, device="cuda")
        self.positions = i32(max_tokens)
        self.q_out = [torch.empty(max_tokens, self.hq, head_dim, dtype=torch.bfloat16, device="cuda")
                      for _ in range(ranks)]
        self.attended = [torch.empty_like(q) for q in self.q_out]
        self.total = [torch.empty(max_tokens, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(ranks)]

    @property
    def lengths(self):
        """[requests] int32 on the GPU: tokens each request holds."""
        return self.len[self.turn]

    def __call__(self, x, new_len):
        """x [tokens, hidden] bfloat16, the new tokens of every request one after the other, padding
        after them; new_len [requests] int32 on the GPU. Returns every rank's copy of the result. Tokens
        of a request that was refused (`refused`, and `refusals` over all steps) and padding come back
        as they were."""
        t, now, then = x.shape[0], self.turn, 1 - self.turn
        if t > self.slots.numel():
            raise ValueError(f"a step holds up to {self.slots.numel()} tokens, got {t}")
        slots, positions = self.slots[:t], self.positions[:t]
        lc.ar_page_tables(self.len[now], new_len, self.pool[now], self.free, self.table, self.len[then],
                          self.q_start, slots, positions, self.pool[then], self.refused, self.page)
        self.turn = then
        torch.maximum(self.refusals, self.refused, out=self.refusals)
        xs = [x] * self.ranks
        for layer in range(self.layers):
            partial = []
            for r in range(self.ranks):
                qkv = xs[r] @ self.w_in[layer][r]
                q, k, v = (y.view(t, -1, self.dim) for y in qkv.split(
                    [self.hq * self.dim, self.hkv * self.dim, self.hkv * self.dim], dim=1))
                data, scales = self.cache[layer][r]
                q_out, out = self.q_out[r][:t], self.attended[r][:t]
                lc.ar_kv4_norm_rope_append(self.kv, q, k, v, q_out, positions, self.cos_sin, slots, data,
                                           scales, self.q_norm, self.k_norm)
                lc.ar_kv4_attention(self.kv, q_out, data, scales, self.table, self.len[then],
                                    self.q_start, out)
                partial.append(out.view(t, -1) @ self.w_out[layer][r])
            total = [y[:t] for y in self.total]
            lc.ar_allreduce(self.sum, partial, total, t * self.hidden, lc.AR_ALGO_AUTO)
            xs = [a + b for a, b in zip(xs, total)]
        # Tokens without a position were attended for with what q_out held before.
        placed = positions[:, None] >= 0
        return [torch.where(placed, y, x) for y in xs]

    def close(self):
        torch.cuda.synchronize()
        lc.ar_check(self.sum)
        lc.ar_destroy(self.sum)
        lc.ar_kv4_destroy(self.kv)


def main(argv=None) -> None:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--ranks", type=int, default=4)
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--requests", type=int, default=16)
    p.add_argument("--prompt", type=int, default=300, help="tokens of the longest prompt")
    p.add_argument("--steps", type=int, default=32, help="decode steps after the prompts")
    a = p.parse_args(argv)
    prompts = [1 + (a.prompt - 1) * (i + 1) // a.requests for i in range(a.requests)]
    run = DecodeStep(a.ranks, a.layers, a.requests, a.prompt + a.steps, sum(prompts))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def tokens(n):
        return torch.randn(n, run.hidden, device="cuda", generator=g).bfloat16()

    run(tokens(sum(prompts)), torch.tensor(prompts, dtype=torch.int32, device="cuda"))
    one = torch.ones(a.requests, dtype=torch.int32, device="cuda")
    x = tokens(a.requests)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(a.steps):
        xs = run(x, one)
        x = xs[0]
    torch.cuda.synchronize()
    us = (time.perf_counter() - start) / max(1, a.steps) * 1e6
    if any(not torch.equal(y, xs[0]) for y in xs):
        raise AssertionError("the ranks' results differ")
    if int(run.refusals.sum()) or run.lengths.tolist() != [n + a.steps for n in prompts]:
        raise AssertionError("a request was refused")
    run.close()
    print(f"{a.ranks} ranks, {a.layers} layers, {a.requests} requests of up to {a.prompt} tokens: "
          f"{us:.1f} us a decode step (all ranks on one GPU, one after another)")


if __name__ == "__main__":
    main()
