"""Plain 64-bit forms of the decode operators on the CPU, for the tests: written from the
definitions in include/ar_decode.h, one loop at a time."""

from __future__ import annotations

import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
# Relative error of one rounding to a type (half a step).
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def page_tables(cached, new, pool, free, table, ntokens, page):
    """(table, kv_len, q_start, slots, positions, pool_out, refused) as lists."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    head, end = max(pool[0], 0), min(pool[1], len(free))
    avail = max(0, end - head)
    taken = wanted = at = 0
    kv, q_start, refused = [], [], []
    slots, positions = [-1] * ntokens, [-1] * ntokens
    for b, (c, n) in enumerate(zip(cached, new)):
        q_start.append(min(at, ntokens))
        have, last = -(-c // page), -(-(c + n) // page)
        fits = c >= 0 and n >= 0 and last <= width and at + max(n, 0) <= ntokens and c + n < 2 ** 31
        need = last - have if fits else 0
        if fits and need > 0:
            fits = wanted + need <= avail
        if fits:
            for j in range(need):
                table[b][have + j] = free[head + wanted + j]
            if need:
                taken = wanted + need
            for i in range(n):
                pos = c + i
                entry = table[b][pos // page]
                positions[at + i] = pos
                slots[at + i] = entry * page + pos % page if entry >= 0 else -1
        wanted += need
        kv.append(c + n if fits else max(c, 0))
        refused.append(0 if fits else 1)
        at += max(n, 0)
    q_start.append(min(at, ntokens))
    return table, kv, q_start, slots, positions, [pool[0] + taken, pool[1]], refused


def norm_rope(x, weight, cos_sin, positions, eps, interleaved):
    """x [T, H, D] of any type -> float64, before the one rounding."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
    if cos_sin is None:
        return y
    rot = cos_sin.shape[1]
    half = rot // 2
    out = y.clone()
    for t in range(x.shape[0]):
        p = int(positions[t])
        if p < 0:
            continue
        if p >= cos_sin.shape[0]:
            out[t] = math.nan
            continue
        c, s = cos_sin[p, :half].double(), cos_sin[p, half:].double()
        a = slice(0, rot, 2) if interleaved else slice(0, half)
        b = slice(1, rot, 2) if interleaved else slice(half, rot)
        out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
        out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
    return out


def quantise(x):
    """(codes [..., D] int64, scale bytes [..., D/32] int64) of rows of binary32 values."""
    y = x.double().reshape(*x.shape[:-1], -1, 32)
    bad = ~torch.isfinite(y).all(-1)
    y = torch.where(bad[..., None], 0.0, y)
    most = y.abs().amax(-1)
    e = torch.full(most.shape, -126, dtype=torch.int64)
    for k in range(-126, 125):  # the smallest power of two that the largest is within six times of
        e = torch.where(most > 6.0 * 2.0 ** k, torch.full_like(e, k + 1), e)
    a = (y / torch.exp2(e.double())[..., None]).abs()
    # the nearest value; at a tie the even code
    dist = (a[..., None] - E2M1).abs()
    odd = torch.arange(8) % 2
    code = (dist * 4 + odd * 1e-9).argmin(-1)
    code = torch.where(torch.signbit(y), code + 8, code)
    code = torch.where(bad[..., None], 0, code)
    return code.reshape(x.shape), torch.where(bad, 255, e + 127)


def dequantise(code, scale):
    v = E2M1[code % 8] * torch.where(code >= 8, -1.0, 1.0).double()
    s = torch.exp2(scale.double() - 127)
    s = torch.where(scale > 252, math.nan, s)
    return (v.reshape(*code.shape[:-1], -1, 32) * s[..., None]).reshape(code.shape)


def pack_row(data, scales, page_size, slot, head, which, code, scale):
    """One row's codes and scales into CPU cache tensors (in place)."""
    pg, off = slot // page_size, slot % page_size
    d = code.numel()
    b = (code[0::2] | (code[1::2] << 4)).to(torch.uint8)
    area = data[pg, head, which]
    if which == 0:
        area.view(page_size, d // 2)[off] = b
    else:
        area.view(page_size // 4, d // 8, 4, 4)[off // 4, :, off % 4] = b.view(d // 8, 4)
    scales[pg, head, which, :, off] = scale.to(torch.uint8)


def unpack(data, scales, page_size):
    """(K, V) [pages, heads, P, D] in float64 of a whole CPU cache."""
    pages, heads = data.shape[:2]
    d = data.shape[-1] * 2 // page_size
    out = []
    for which in (0, 1):
        x = data[:, :, which]
        if which == 0:
            x = x.reshape(pages, heads, page_size, d // 2)
        else:
            x = x.reshape(pages, heads, page_size // 4, d // 8, 4, 4).transpose(3, 4)
            x = x.reshape(pages, heads, page_size, d // 2)
        x = x.long()
        code = torch.stack([x & 15, x >> 4], dim=-1).reshape(pages, heads, page_size, d)
        out.append(dequantise(code, scales[:, :, which].transpose(2, 3).long()))
    return out


def attention(q, k_pages, v_pages, table, kv_len, q_start, page_size, scale, window):
    """(out, lse, bound) [T, Hq, D], [T, Hq], [T, Hq, D]: float64 results and the errors that the
    kernel's roundings allow.

    The bound follows the kernel's arithmetic with half = the type's rounding and A = sum p |v| / l:
    probabilities rounded once (half A; 2^-24 A for binary32), sums of n binary32 terms
    (n 2^-23 A), scores off by delta = scale sum |q k| D 2^-23 + 4 |s| 2^-24, which moves a
    probability and the sum by at most that part (2 delta A), the exponential's own error
    (2^-21 A), and the result's rounding (half |o|). Probabilities below binary32's smallest normal
    value, 2^-126 of a reference that trails the row's maximum by at most 2^8, are zero: n 2^-118
    of the largest value (a part in 10^35, seen only where every larger probability meets a value
    that is exactly zero)."""
    t, hq, d = q.shape
    heads = k_pages.shape[1]
    group = hq // heads
    half = HALF[q.dtype]
    out = torch.full((t, hq, d), math.nan, dtype=torch.float64)
    lse = torch.full((t, hq), math.nan, dtype=torch.float64)
    bound = torch.zeros(t, hq, d, dtype=torch.float64)
    lse_bound = torch.zeros(t, hq, dtype=torch.float64)
    pages = k_pages.shape[0]
    for b in range(len(kv_len)):
        m, n = int(q_start[b + 1]) - int(q_start[b]), max(int(kv_len[b]), 0)
        n_room = min(n, table.shape[1] * page_size)
        ids = table[b].long()[:-(-n_room // page_size)]
        ok = ((ids >= 0) & (ids < pages)).repeat_interleave(page_size)[:n_room]
        ids = ids.clamp(0, pages - 1)
        k = k_pages[ids].transpose(0, 1).reshape(heads, -1, d)[:, :n_room]
        v = v_pages[ids].transpose(0, 1).reshape(heads, -1, d)[:, :n_room]
        pos = torch.arange(n_room)
        for i in range(m):
            p = n - m + i
            see = ok & (pos <= p)
            if window > 0:
                see = see & (pos > p - window)
            row = int(q_start[b]) + i
            if not bool(see.any()):
                out[row], lse[row] = 0.0, -math.inf
                continue
            kk, vv = k[:, see], v[:, see]
            qq = q[row].double().view(heads, group, d)
            s = qq @ kk.transpose(1, 2) * scale  # [heads, group, n]
            size = (qq.abs() @ kk.abs().transpose(1, 2)) * abs(scale)
            delta = (size * d * 2.0 ** -23 + 4 * s.abs() * 2.0 ** -24).amax(-1, keepdim=True)
            top = s.amax(-1, keepdim=True)
            e = torch.exp(s - top)
            l = e.sum(-1, keepdim=True)
            prob = e / l
            out[row] = (prob @ vv).reshape(hq, d)
            lse[row] = (top + torch.log(l)).reshape(hq)
            a = prob @ vv.abs()
            cnt = kk.shape[1]
            rel = half + (cnt + 64) * 2.0 ** -23 + 2 * delta + 2.0 ** -21
            bound[row] = (rel * a).reshape(hq, d) + half * out[row].abs()
            bound[row] += cnt * 2.0 ** -118 * float(vv.nan_to_num(nan=0.0).abs().max())
            lse_bound[row] = (delta.reshape(hq) + (cnt + 64) * 2.0 ** -23
                              + 4 * 2.0 ** -24 * lse[row].abs())
    return out, lse, bound, lse_bound
