"""Plain 64-bit forms of the serving operators on the CPU, for the tests: written from the definitions in
include/ar_serving.h, one loop at a time."""

from __future__ import annotations

import math

import torch

from tests import decode_ref as R

BLOCK = 16


def _e4m3():
    """The 256 values that codes stand for."""
    out = []
    for code in range(256):
        p, f = (code >> 3) & 15, (code & 7) / 8
        y = f * 2.0 ** -6 if p == 0 else (1 + f) * 2.0 ** (p - 7)
        if code & 127 == 127:
            y = math.nan
        out.append(-y if code >= 128 else y)
    return torch.tensor(out, dtype=torch.float64)


E4M3 = _e4m3()


def exponent(most):
    """The smallest e, -100 to 119, with most <= 448 * 2^e."""
    e = -100
    while e < 119 and most > 448.0 * 2.0 ** e:
        e += 1
    return e


def rounded(y, e):
    """float64 values to the nearest that a code at scale 2^e stands for, ties to the even code."""
    a = (y.abs() / 2.0 ** e).clamp(max=448.0)
    grid = E4M3[:127]
    i = torch.searchsorted(grid, a.contiguous()).clamp(1, 126)  # grid[i-1] < a <= grid[i]
    lo, hi = grid[i - 1], grid[i]
    up = (hi - a < a - lo) | ((hi - a == a - lo) & (i % 2 == 0))
    r = torch.where(up, hi, lo) * 2.0 ** e
    r = torch.where(torch.isfinite(y), torch.copysign(r, y), math.nan)
    return r


class Cache:
    """The values [pages, heads, 2, P, D] and scale exponents [pages, heads, P / 16, 2] of a cache."""

    def __init__(self, pages, heads, d, page):
        self.page = page
        self.values = torch.zeros(pages, heads, 2, page, d, dtype=torch.float64)
        self.e = torch.zeros(pages, heads, page // BLOCK, 2, dtype=torch.int64)

    def append(self, k, v, slots):
        """Rows k, v [T, heads, D] to `slots`, run by run."""
        pages, heads = self.values.shape[:2]
        slots = [s if 0 <= s < pages * self.page else -1 for s in slots]
        runs = {}
        for t, s in enumerate(slots):
            if s >= 0:
                runs.setdefault((s // BLOCK, s - t), []).append(t)
        for (block, _), run in runs.items():
            pg, b = block * BLOCK // self.page, block % (self.page // BLOCK)
            o = [slots[t] % BLOCK for t in run]
            for h in range(heads):
                for which, x in ((0, k), (1, v)):
                    y = x[run, h].double()
                    fine = y[torch.isfinite(y)]
                    e = exponent(float(fine.abs().max()) if fine.numel() else 0.0)
                    area = self.values[pg, h, which, b * BLOCK:(b + 1) * BLOCK]
                    if o[0] > 0:
                        had = min(max(int(self.e[pg, h, b, which]), -100), 119)
                        if e > had:
                            area.copy_(rounded(area, e))
                        e = max(e, had)
                    area[o] = rounded(y, e)
                    self.e[pg, h, b, which] = e


def unpack(data, scales, d):
    """([pages, heads, 2, P, D] values, [pages, heads, P / 16, 2] exponents) of CPU tensors."""
    pages, heads, _, size = data.shape
    page = size // d
    k = data[:, :, 0].view(pages, heads, page, d)
    v = data[:, :, 1].view(pages, heads, page // 4, d, 4).transpose(3, 4).reshape(pages, heads, page, d)
    x = E4M3[torch.stack([k, v], dim=2).long()]
    e = scales.long() - 127
    size = torch.exp2(e.clamp(-100, 119).double()).transpose(2, 3).repeat_interleave(BLOCK, dim=3)
    return x * size[..., None], e


def prompt_attention(q, k, v, q_start, scale, window):
    """(out, lse, bounds) over packed prompts: those of a request are its own attention over its own tokens."""
    t, hq, d = q.shape
    res = [torch.full((t, hq, d), math.nan, dtype=torch.float64), torch.full((t, hq), math.nan, dtype=torch.float64),
           torch.zeros(t, hq, d, dtype=torch.float64), torch.zeros(t, hq, dtype=torch.float64)]
    at = [min(max(int(x), 0), t) for x in q_start]
    for b in range(len(at) - 1):
        lo, hi = at[b], max(at[b], at[b + 1])
        if hi == lo:
            continue
        n = hi - lo
        pages = [x[lo:hi].double().transpose(0, 1)[None] for x in (k, v)]
        got = R.attention(q[lo:hi], *pages, torch.zeros(1, 1, dtype=torch.int32), [n], [0, n], n, scale, window)
        for x, y in zip(res, got):
            x[lo:hi] = y
    return res


# ------------------------------------------------------------------ pages


def pages_for(n, page):
    return -(-n // page) if n > 0 else 0


def fork(src, dst, kv_len, table, shares, pool, free, page):
    """(table, shares, kv_len_out, pool_out, copy_src, copy_dst, refused), lists throughout."""
    table, shares, out = [list(r) for r in table], list(shares), list(kv_len)
    width = len(table[0]) if table else 0
    head, end = max(pool[0], 0), min(pool[1], len(free))
    taken = wanted = 0
    copies, refused, seen = [], [], set()
    for s, d in zip(src, dst):
        fits = 0 <= s < len(kv_len) and 0 <= d < len(kv_len) and s != d and d not in seen
        if 0 <= d < len(kv_len):
            seen.add(d)
        fits = fits and kv_len[d] == 0 and kv_len[s] >= 0 and pages_for(kv_len[s], page) <= width
        need = fits and kv_len[s] % page != 0
        if need:
            fits = wanted < max(0, end - head)
            wanted += 1
        copy = (-1, -1)
        if fits:
            whole = kv_len[s] // page
            for j in range(whole):
                table[d][j] = table[s][j]
                if 0 <= table[s][j] < len(shares):
                    shares[table[s][j]] += 1
            if need:
                table[d][whole] = free[head + wanted - 1]
                copy = (table[s][whole], table[d][whole])
                taken = wanted
            out[d] = kv_len[s]
        copies.append(copy)
        refused.append(0 if fits else 1)
    return (table, shares, out, [head + taken, pool[1]], [c[0] for c in copies], [c[1] for c in copies], refused)


def free_pages(requests, kv_len, table, shares, pool, free, page):
    """(shares, free, kv_len_out, pool_out)."""
    shares, free, out = list(shares), list(free), list(kv_len)
    width = len(table[0]) if table else 0
    gone = set()
    for b in dict.fromkeys(r for r in requests if 0 <= r < len(kv_len)):
        for j in range(min(pages_for(kv_len[b], page), width)):
            p = table[b][j]
            if 0 <= p < len(shares):
                if shares[p] <= 0:
                    gone.add(p)
                shares[p] -= 1
        out[b] = 0
    for p in gone:
        shares[p] = 0
    first = min(max(pool[0], 0), len(free))
    start = first - len(gone)
    for k, p in enumerate(sorted(gone)):
        if start + k >= 0:
            free[start + k] = p
    return shares, free, out, [max(start, 0), pool[1]]


def compact(kv_len, table, shares, page, nmoves):
    """(table, shares, pool_out, move_src, move_dst)."""
    width = len(table[0]) if table else 0
    held = set()
    for b, n in enumerate(kv_len):
        held |= {p for p in table[b][:min(pages_for(n, page), width)] if 0 <= p < len(shares)}
    n = len(held)
    src = sorted(p for p in held if p >= n)
    dst = [p for p in range(n) if p not in held]
    to = dict(zip(src, dst))
    out = [[to.get(p, p) if j < pages_for(kv_len[b], page) else -1 for j, p in enumerate(row)]
           for b, row in enumerate(table)]
    counts = [0] * len(shares)
    for p in held:
        counts[to.get(p, p)] = shares[p]
    pad = [-1] * (nmoves - len(src))
    return out, counts, [n, len(shares)], src + pad, dst[:len(src)] + pad


# ------------------------------------------------------------------ many rows, on any device


def dense_attention(q, k, v, scale, window):
    """(out, lse, bound, lse_bound) of one request in 64 bits, all rows of a head at once: q [m, hq, d] in its type
    are the last m of the n positions of k, v [n, hkv, d] (values in any type). Definition and bounds are those of
    decode_ref.attention; what is not finite among the values reaches the rows that see it."""
    m, hq, d = q.shape
    n, heads = k.shape[0], k.shape[1]
    group, half, dev = hq // heads, R.HALF[q.dtype], q.device
    out, bound = (torch.zeros(m, hq, d, dtype=torch.float64, device=dev) for _ in range(2))
    lse, lse_bound = (torch.zeros(m, hq, dtype=torch.float64, device=dev) for _ in range(2))
    pos = torch.arange(n - m, n, device=dev).repeat_interleave(group)[:, None]  # a row of s a token and head of the group
    t = torch.arange(n, device=dev)[None]
    see = t <= pos
    if window > 0:
        see &= t > pos - window
    cnt = see.sum(-1, keepdim=True)
    seen = see.double()
    for h in range(heads):
        x = q[:, h * group:(h + 1) * group].double().reshape(m * group, d)
        kt = k[:, h].double().t().contiguous()
        vv = v[:, h].double()
        s = x @ kt * scale
        delta = ((x.abs() @ kt.abs()) * (abs(scale) * d * 2.0 ** -23) + 4 * s.abs() * 2.0 ** -24)
        delta = delta.masked_fill(~see, 0.0).amax(-1, keepdim=True)
        s = s.masked_fill(~see, -math.inf)
        top = s.amax(-1, keepdim=True)
        nothing = cnt == 0
        e = torch.exp(s - top.masked_fill(nothing, 0.0))
        l = e.sum(-1, keepdim=True)
        prob = e / l.masked_fill(nothing, 1.0)
        finite = vv.nan_to_num(nan=0.0, posinf=0.0, neginf=0.0)
        o = prob @ finite
        rel = half + (cnt + 64) * 2.0 ** -23 + 2 * delta + 2.0 ** -21
        b = rel * (prob @ finite.abs()) + half * o.abs() + cnt * 2.0 ** -118 * finite.abs().max()
        if not bool(torch.isfinite(vv).all()):
            up = seen @ (torch.isnan(vv) | (vv == math.inf)).double() > 0
            down = seen @ (torch.isnan(vv) | (vv == -math.inf)).double() > 0
            o = o + torch.where(up, math.inf, 0.0)
            o = o - torch.where(down, math.inf, 0.0)
        at = slice(h * group, (h + 1) * group)
        out[:, at], bound[:, at] = o.view(m, group, d), b.view(m, group, d)
        y = top + torch.log(l)
        lse[:, at] = y.view(m, group)
        lse_bound[:, at] = (delta + (cnt + 64) * 2.0 ** -23 + 4 * 2.0 ** -24 * y.abs()).view(m, group)
    return out, lse, bound, lse_bound
