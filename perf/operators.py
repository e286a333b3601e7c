"""Cases of the decode operators: page tables, per-head norm with rotation, the 4-bit paged cache
and the attention that reads it.

Where ``own`` is false, ``run`` computes an operator with elementary torch operations; where it is
true, it makes the calls of ``latency_collectives_amd`` that a serving program makes.

The 4-bit cache, as both sides hold it: ``data`` uint8 [pages, heads, 2, P * D / 2] and ``scales``
uint8 [pages, heads, 2, D / 32, P] (index 0 of the third axis is K, 1 is V). A K row is D / 2 bytes,
element 2 i in the low four bits of byte i. V rows are interleaved by four tokens: the bytes of a
page are [P / 4][D / 8][4 tokens][4 bytes]. A code is e2m1 (sign, two exponent bits, one mantissa
bit), a scale byte s stands for 2^(s - 127), 255 for NaN.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_GOLD = 0.6180339887498949


# ------------------------------------------------------------------ cases


def listed():
    return [
        # One decode step of a small batch: every request grows by one token. Latency counts.
        {"name": "tables_decode", "kind": "tables", "b": 32, "new": 1, "kv": 4096, "page": 16},
        # A large mixed batch: decodes and prompt chunks, a thousand requests.
        {"name": "tables_mixed", "kind": "tables", "b": 1000, "new": 64, "kv": 16384, "page": 32},
        # One token of one tensor-parallel rank: 8 query heads, 1 key head.
        {"name": "rope_token", "kind": "rope", "dtype": "bf16", "t": 1, "hq": 8, "hkv": 1, "d": 128,
         "rot": 128, "inter": False, "norm": True},
        # A prompt chunk of the whole layer's heads, an odd number of tokens.
        {"name": "rope_prompt", "kind": "rope", "dtype": "bf16", "t": 8191, "hq": 32, "hkv": 8,
         "d": 128, "rot": 128, "inter": False, "norm": True},
        # Binary32, adjacent pairs, half of the head rotated.
        {"name": "rope_f32_partial", "kind": "rope", "dtype": "f32", "t": 1000, "hq": 12, "hkv": 4,
         "d": 96, "rot": 48, "inter": True, "norm": True},
        # Norm, rotation and the cache's new rows of a decode step over 64 requests.
        {"name": "fused_decode", "kind": "fused", "dtype": "bf16", "t": 64, "hq": 8, "hkv": 1,
         "d": 128, "rot": 128, "inter": False, "page": 16},
        # A prompt's keys and values into the cache.
        {"name": "append_prompt", "kind": "append", "dtype": "bf16", "t": 5001, "hkv": 8, "d": 128,
         "page": 32},
        # One request, one rank's heads: the smallest attention of a decode step.
        {"name": "attn_single", "kind": "attn", "dtype": "bf16", "b": 1, "new": 1, "kv": 2000,
         "hq": 8, "hkv": 1, "d": 128, "page": 16, "window": 0},
        # An ordinary decode batch of ragged lengths.
        {"name": "attn_decode", "kind": "attn", "dtype": "bf16", "b": 64, "new": 1, "kv": 8192,
         "hq": 32, "hkv": 8, "d": 128, "page": 16, "window": 0},
        # Long contexts.
        {"name": "attn_long", "kind": "attn", "dtype": "bf16", "b": 8, "new": 1, "kv": 131072,
         "hq": 64, "hkv": 8, "d": 128, "page": 64, "window": 0},
        # Chunks of prompts against what is cached already: compute-bound.
        {"name": "attn_chunk", "kind": "attn", "dtype": "bf16", "b": 2, "new": 2048, "kv": 12288,
         "hq": 32, "hkv": 8, "d": 128, "page": 32, "window": 0},
        # Binary32, a small head, several tokens a request (drafted ones), a sliding window.
        {"name": "attn_f32_window", "kind": "attn", "dtype": "f32", "b": 19, "new": 5, "kv": 5000,
         "hq": 16, "hkv": 4, "d": 64, "page": 16, "window": 1024},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tables", "rope", "fused", "append", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 96, 128, 128, 192, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    if kind == "tables":
        return {"kind": kind, "b": _log(rng, 1, 2048), "new": _log(rng, 1, 64),
                "kv": _log(rng, 16, 16384), "page": page}
    rot = rng.choice([d, d, d // 2])
    if kind == "rope":
        t = _log(rng, 1, 8191 * 40 * 128 // ((hq + hkv) * d * (2 if dtype == "f32" else 1)))
        return {"kind": kind, "dtype": dtype, "t": min(t, 8191), "hq": hq, "hkv": hkv, "d": d,
                "rot": rot, "inter": rng.random() < 0.4, "norm": rng.random() < 0.8}
    if kind == "fused":
        return {"kind": kind, "dtype": dtype, "t": _log(rng, 1, 1500), "hq": hq, "hkv": hkv, "d": d,
                "rot": rot, "inter": rng.random() < 0.4, "page": page}
    if kind == "append":
        return {"kind": kind, "dtype": dtype, "t": _log(rng, 1, 5000), "hkv": hkv, "d": d,
                "page": page}
    new = rng.choice([1, 1, 1, 2, 4, _log(rng, 8, 700)])
    kv = _log(rng, new, 65536 if new == 1 else 12000)
    most = int(6e6 if new == 1 else 6e7 / (new * hq // hkv))
    b = _log(rng, 1, max(1, min(200, most // max(1, kv * hkv))))
    return {"kind": kind, "dtype": dtype, "b": b, "new": new, "kv": kv, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)])}


def _new_lens(c):
    """Tokens each request brings: decode steps bring one, others 1 .. new."""
    return [1 + int((c["new"] - 1) * ((i * _GOLD + 1.0) % 1.0 if i else 1.0)) for i in range(c["b"])]


def _kv_lens(c):
    """Length of each request with its new tokens: the first has the most, others are ragged."""
    new = _new_lens(c)
    lens = [c["kv"] if i == 0 else 1 + int((c["kv"] - 1) * ((i * _GOLD + 0.3) % 1.0))
            for i in range(c["b"])]
    return [max(n, m) for n, m in zip(lens, new)]


def _pages(c):
    return sum(-(-n // c["page"]) for n in _kv_lens(c))


def work(c):
    es = 4 if c.get("dtype") == "f32" else 2
    if c["kind"] == "tables":
        new = _new_lens(c)
        fresh = _pages(c) - sum(-(-(n - m) // c["page"]) for n, m in zip(_kv_lens(c), new))
        return {"bytes": c["b"] * 20 + sum(new) * 12 + fresh * 8, "flops": 0}
    if c["kind"] == "rope":
        return {"bytes": c["t"] * ((c["hq"] + c["hkv"]) * c["d"] * es * 2 + c["rot"] * 4 + 4),
                "flops": 8 * c["t"] * (c["hq"] + c["hkv"]) * c["d"]}
    if c["kind"] in ("append", "fused"):  # into the cache, and the new rows read back as values
        row = c["d"] * es + 2 * (c["d"] // 2 + c["d"] // 32) + c["d"] * 2
        n = c["t"] * (2 * c["hkv"] * row + 16)
        if c["kind"] == "fused":
            n += c["t"] * (c["hq"] * c["d"] * es * 2 + c["rot"] * 4 + 4)
        return {"bytes": n, "flops": 8 * c["t"] * c["hkv"] * c["d"]}
    new, lens, seen, read = _new_lens(c), _kv_lens(c), 0, 0
    for n, m in zip(lens, new):
        if c["window"]:
            seen += sum(min(c["window"], n - m + i + 1) for i in range(m))
            read += min(n, c["window"] + m - 1)
        else:
            seen += m * (n - m) + m * (m + 1) // 2
            read += n
    t = sum(new)
    return {"bytes": read * c["hkv"] * 2 * (c["d"] // 2 + c["d"] // 32)
            + t * c["hq"] * (2 * c["d"] * es + 4) + 4 * (_pages(c) + 3 * c["b"]),
            "flops": 4 * seen * c["hq"] * c["d"]}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _cos_sin(rows, rot):
    """[rows, rot] binary32: the cosines of rot / 2 angles, then their sines."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _handle(c):
    """What a serving program keeps for caches of this geometry."""
    if not own:
        return None
    import latency_collectives_amd as lc

    key = (c["hkv"], c["d"], c["page"])
    if key not in _handles:
        _handles[key] = lc.ar_kv4_create(*key)
    return _handles[key]


_handles = {}


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": c, "kind": c["kind"]}
    if c["kind"] == "tables":
        new, lens, page = _new_lens(c), _kv_lens(c), c["page"]
        had = [n - m for n, m in zip(lens, new)]
        width = max(-(-n // page) for n in lens)
        pages = _pages(c) + 8
        perm = torch.randperm(pages, device="cuda", generator=g).int()
        table = torch.full((c["b"], width), -1, dtype=torch.int32, device="cuda")
        at = 0
        counts = _i32([-(-n // page) for n in had])
        held = torch.arange(width, device="cuda")[None, :] < counts[:, None]
        at = int(counts.sum())
        table[held] = perm[:at]
        cap = sum(new) + 7  # a step's buffers are padded to a fixed size
        s.update(cached=_i32(had), new=_i32(new), pool=_i32([0, pages - at]), free=perm[at:].contiguous(),
                 table=table, page=page, cap=cap, width=width,
                 kv_len=torch.empty(c["b"], dtype=torch.int32, device="cuda"),
                 q_start=torch.empty(c["b"] + 1, dtype=torch.int32, device="cuda"),
                 slots=torch.empty(cap, dtype=torch.int64, device="cuda"),
                 positions=torch.empty(cap, dtype=torch.int32, device="cuda"),
                 pool_out=torch.empty(2, dtype=torch.int32, device="cuda"),
                 refused=torch.empty(c["b"], dtype=torch.int32, device="cuda"))
        return s
    dt = _TYPES[c["dtype"]]
    if c["kind"] in ("rope", "fused", "append"):
        t, hkv, d = c["t"], c["hkv"], c["d"]
        hq = c.get("hq", 0)
        # the projection's output: q, k and v of a token side by side
        qkv = torch.randn(t, (hq + 2 * hkv) * d, device="cuda", generator=g).to(dt)
        q, k, v = (x.view(t, -1, d) for x in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
        s.update(q=q, k=k, v=v)
        if c["kind"] != "append":
            rows = 32768
            s.update(cos_sin=_cos_sin(rows, c["rot"]), eps=1e-6, inter=c["inter"],
                     positions=torch.randint(0, rows, (t,), device="cuda", generator=g).int(),
                     q_out=torch.empty(t, hq, d, dtype=dt, device="cuda"), wq=None, wk=None)
            if c.get("norm", True):
                s.update(wq=(1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(dt),
                         wk=(1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(dt))
        if c["kind"] == "rope":
            s["k_out"] = torch.empty(t, hkv, d, dtype=dt, device="cuda")
            return s
        page = c["page"]
        pages = -(-t // page) + 5
        # new rows go to random places, some tokens are padding
        slots = torch.randperm(pages * page, device="cuda", generator=g)[:t]
        slots[t // 3 + 1::97] = -1
        s.update(slots=slots, page=page, handle=_handle(c),
                 data=torch.zeros(pages, hkv, 2, page * d // 2, dtype=torch.uint8, device="cuda"),
                 scales=torch.zeros(pages, hkv, 2, d // 32, page, dtype=torch.uint8, device="cuda"),
                 k_read=torch.empty(t, hkv, d, dtype=torch.bfloat16, device="cuda"),
                 v_read=torch.empty(t, hkv, d, dtype=torch.bfloat16, device="cuda"))
        return s
    # attention over a cache of quantised normal values
    new, lens, page, d, hkv = _new_lens(c), _kv_lens(c), c["page"], c["d"], c["hkv"]
    pages = _pages(c) + 3
    width = max(-(-n // page) for n in lens)
    stock = min(pages, 257)
    data = torch.zeros(stock, hkv, 2, page * d // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(stock, hkv, 2, d // 32, page, dtype=torch.uint8, device="cuda")
    rows = torch.randn(2, stock * page, hkv, d, device="cuda", generator=g)
    _put(data, scales, rows[0], rows[1], torch.arange(stock * page, device="cuda"), page)
    pick = torch.randint(0, stock, (pages,), device="cuda", generator=g)
    data, scales = data[pick], scales[pick]
    perm = torch.randperm(pages, device="cuda", generator=g).int()
    table = torch.full((c["b"], width), -1, dtype=torch.int32, device="cuda")
    counts = _i32([-(-n // page) for n in lens])
    table[torch.arange(width, device="cuda")[None, :] < counts[:, None]] = perm[:int(counts.sum())]
    t = sum(new)
    s.update(q=torch.randn(t, c["hq"], d, device="cuda", generator=g).to(dt), data=data, scales=scales,
             table=table, kv_len=_i32(lens), q_start=_i32(_starts(new)), page=page, most=max(new),
             scale=1.0 / math.sqrt(d), window=c["window"], handle=_handle(c),
             out=torch.empty(t, c["hq"], d, dtype=dt, device="cuda"),
             lse=torch.empty(t, c["hq"], dtype=torch.float32, device="cuda"))
    return s


# ------------------------------------------------------------------ plain forms

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _encode(x):
    """Codes [..., D] and scale bytes [..., D / 32] of x [..., D]: a group of 32 takes the smallest
    power of two with no value over 6 of it; codes are nearest, ties to the even one."""
    y = x.double().unflatten(-1, (-1, 32))
    most = y.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(most)  # most = m 2^e with 0.5 <= m < 1, and 6 = 0.75 * 2^3
    e = torch.where(most > 0, e - 3 + (m > 0.75), torch.full_like(e, -126)).clamp(min=-126)
    y = torch.ldexp(y, -e)
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
            + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())
    code = (code + 8 * torch.signbit(y).int()).flatten(-2).to(torch.uint8)
    return code, (e + 127).squeeze(-1).to(torch.uint8)


def _put(data, scales, k, v, slots, page):
    """Writes rows k, v [T, heads, D] at `slots` (negative: nowhere)."""
    t, heads, d = k.shape
    live = slots >= 0
    at, k, v = slots[live], k[live], v[live]
    pg, off = at // page, at % page
    kc, ks = _encode(k)
    vc, vs = _encode(v)
    kb, vb = (x[..., 0::2] | (x[..., 1::2] << 4) for x in (kc, vc))
    pages = data.shape[0]
    data[:, :, 0].unflatten(-1, (page, d // 2))[pg, :, off] = kb
    data[:, :, 1].unflatten(-1, (page // 4, d // 8, 4, 4))[pg, :, off // 4, :, off % 4] = vb.view(-1, heads, d // 8, 4)
    sc = scales.view(pages, heads, 2, d // 32, page)
    sc[:, :, 0][pg, :, :, off] = ks
    sc[:, :, 1][pg, :, :, off] = vs


def _lut():
    v = torch.tensor(_E2M1, device="cuda")
    v = torch.cat([v, -v])
    b = torch.arange(256, device="cuda")
    return torch.stack([v[b & 15], v[b >> 4]], dim=1)


def _decode(data, scales, page, d):
    """K and V [n, heads, P, D] in binary32 of whole pages data [n, heads, 2, ...]."""
    n, heads = data.shape[:2]
    lut = _lut()
    k = data[:, :, 0].reshape(n, heads, page, d // 2)
    v = data[:, :, 1].reshape(n, heads, page // 4, d // 8, 4, 4).transpose(3, 4).reshape(n, heads, page, d // 2)
    x = torch.exp2(scales.float() - 127).transpose(-1, -2)  # [n, heads, 2, P, D / 32]
    k = (lut[k.int()].view(n, heads, page, d // 32, 32) * x[:, :, 0, :, :, None]).flatten(-2)
    v = (lut[v.int()].view(n, heads, page, d // 32, 32) * x[:, :, 1, :, :, None]).flatten(-2)
    return k, v


def _get(data, scales, slots, page, d):
    """Rows [T, heads, D] of K and V at `slots`, zeros where the slot is negative."""
    at = slots.clamp(min=0)
    pg, off = at // page, at % page
    k, v = _decode(data, scales, page, d)
    live = (slots >= 0)[:, None, None]
    return tuple(torch.where(live, x[pg, :, off], 0.0).to(torch.bfloat16) for x in (k, v))


def _norm_rope(x, w, cs, positions, eps, inter, wide):
    """Per-head RMS norm (where there is a weight) and rotation of x [T, H, D], in `wide`."""
    y = x.to(wide)
    if w is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * w.to(wide)
    rot = cs.shape[1]
    row = cs[positions.long()].to(wide)[:, None, :]
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])
    p, q = a * c - b * s, b * c + a * s
    p = torch.stack([p, q], dim=-1).flatten(-2) if inter else torch.cat([p, q], dim=-1)
    return torch.cat([p, y[..., rot:]], dim=-1).to(x.dtype)


def _plain_tables(s):
    page, b = s["page"], s["cached"].numel()
    had, new = s["cached"].long(), s["new"].long()
    start = torch.cat([new.new_zeros(1), new.cumsum(0)])
    first, last = (had + page - 1) // page, (had + new + page - 1) // page
    need = last - first
    base = need.cumsum(0) - need
    fits = (need == 0) | (base + need <= s["pool"][1] - s["pool"][0])
    fits = fits & (last <= s["width"]) & (start[1:] <= s["cap"])
    col = torch.arange(s["width"], device="cuda")
    fresh = (col >= first[:, None]) & (col < last[:, None]) & fits[:, None]
    which = (s["pool"][0] + base[:, None] + col - first[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][which], s["table"])
    i = torch.arange(s["cap"], device="cuda")
    r = torch.searchsorted(start[1:], i, right=True).clamp(max=b - 1)
    live = (i < start[-1]) & fits[r]
    pos = had[r] + i - start[r]
    entry = table[r, (pos // page).clamp(0, s["width"] - 1)].long()
    used = torch.where(fits & (need > 0), base + need, 0).amax()
    return {"table": table, "kv_len": torch.where(fits, had + new, had).int(), "q_start": start.int(),
            "slots": torch.where(live, entry * page + pos % page, -1),
            "positions": torch.where(live, pos, -1).int(),
            "pool": torch.stack([s["pool"][0] + used, s["pool"][1]]).int(), "refused": (~fits).int()}


def _plain_attn(s):
    page, d = s["page"], s["q"].shape[2]
    b, width = s["table"].shape
    heads = s["data"].shape[1]
    group = s["q"].shape[1] // heads
    k, v = _decode(s["data"][s["table"].clamp(min=0)].flatten(0, 1),
                   s["scales"][s["table"].clamp(min=0)].flatten(0, 1), page, d)
    # [B, heads, tokens, D]
    k, v = (x.view(b, width, heads, page, d).transpose(1, 2).reshape(b, heads, width * page, d) for x in (k, v))
    start, lens = s["q_start"].long(), s["kv_len"].long()
    new = start[1:] - start[:-1]
    i = torch.arange(s["most"], device="cuda")
    at = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[at].view(b, s["most"], heads, group, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(b, heads, group * s["most"], d), k.transpose(2, 3)) * s["scale"]
    x = x.view(b, heads, group, s["most"], width * page)
    t = torch.arange(width * page, device="cuda")
    pos = (lens - new)[:, None] + i  # [B, new]
    seen = (t <= pos[..., None]) & (t < lens[:, None, None])
    if s["window"]:
        seen = seen & (t > pos[..., None] - s["window"])
    seen = seen[:, None, None]
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, heads, group * s["most"], -1), v).view(b, heads, group, s["most"], d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(b, s["most"], heads * group, d)
    lse = (m + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(b, s["most"], heads * group)
    live = i < new[:, None]
    return {"out": o[live].to(s["q"].dtype), "lse": lse[live]}


def run(s):
    kind = s["kind"]
    if own:
        import latency_collectives_amd as lc

        if kind == "tables":
            lc.ar_page_tables(s["cached"], s["new"], s["pool"], s["free"], s["table"], s["kv_len"],
                              s["q_start"], s["slots"], s["positions"], s["pool_out"], s["refused"],
                              s["page"])
            return {k: s[k] for k in ("table", "kv_len", "q_start", "slots", "positions", "refused")} | {"pool": s["pool_out"]}
        if kind == "rope":
            lc.ar_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["cos_sin"],
                               s["wq"], s["wk"], s["eps"], s["inter"])
            return {"q": s["q_out"], "k": s["k_out"]}
        if kind in ("fused", "append"):
            out = {}
            if kind == "fused":
                lc.ar_kv4_norm_rope_append(s["handle"], s["q"], s["k"], s["v"], s["q_out"],
                                           s["positions"], s["cos_sin"], s["slots"], s["data"],
                                           s["scales"], s["wq"], s["wk"], s["eps"], s["inter"])
                out["q"] = s["q_out"]
            else:
                lc.ar_kv4_append(s["handle"], s["k"], s["v"], s["slots"], s["data"], s["scales"])
            lc.ar_kv4_read(s["handle"], s["slots"], s["data"], s["scales"], s["k_read"], s["v_read"])
            return out | {"k": s["k_read"], "v": s["v_read"]}
        lc.ar_kv4_attention(s["handle"], s["q"], s["data"], s["scales"], s["table"], s["kv_len"],
                            s["q_start"], s["out"], s["lse"], s["scale"], s["window"])
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "tables":
        return _plain_tables(s)
    if kind == "rope":
        return {x: _norm_rope(s[x], s["w" + x], s["cos_sin"], s["positions"], s["eps"], s["inter"], torch.float32)
                for x in ("q", "k")}
    if kind in ("fused", "append"):
        out, k = {}, s["k"]
        if kind == "fused":
            # keys go on to four bits: 64 bits keep their roundings away from the codes' borders
            out["q"] = _norm_rope(s["q"], s["wq"], s["cos_sin"], s["positions"], s["eps"], s["inter"], torch.float32)
            k = _norm_rope(k, s["wk"], s["cos_sin"], s["positions"], s["eps"], s["inter"], torch.float64)
        _put(s["data"], s["scales"], k, s["v"], s["slots"], s["page"])
        k, v = _get(s["data"], s["scales"], s["slots"], s["page"], s["k"].shape[2])
        return out | {"k": k, "v": v}
    return _plain_attn(s)


# ------------------------------------------------------------------ definitions in 64 bits


def _exact_rotated(x, w, s):
    t, h, d = x.shape
    y = x.double()
    if w is not None:
        y = y * torch.rsqrt((y * y).sum(2, keepdim=True) / d + s["eps"]) * w.double()
    rot = s["cos_sin"].shape[1]
    half = rot // 2
    cs = s["cos_sin"].double()[s["positions"].long()]
    z = torch.complex(cs[:, :half], cs[:, half:])[:, None]
    j = torch.arange(half, device="cuda")
    a, b = (2 * j, 2 * j + 1) if s["inter"] else (j, j + half)
    turned = torch.complex(y[..., a], y[..., b]) * z
    out = y.clone()
    out[..., a], out[..., b] = turned.real, turned.imag
    return out


def _exact_stored(x, slots):
    """The values that the cache stands for after rows x are written: the nearest of the 15 values
    of each group, ties to the even code."""
    t, h, d = x.shape
    y = x.double().reshape(t, h, d // 32, 32)
    most = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2((most / 6).clamp(min=2.0 ** -126)))
    e = torch.where(most <= 6 * torch.exp2(e - 1), e - 1, e)  # the logarithm's rounding
    e = torch.where(most > 6 * torch.exp2(e), e + 1, e).clamp(min=-126)
    a = y.abs() / torch.exp2(e)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    r = torch.round(a / step) * step  # torch.round: ties to even, as the codes' last bit is
    r = torch.copysign(r * torch.exp2(e), y).reshape(t, h, d)
    return torch.where((slots >= 0)[:, None, None], r, 0.0)


def exact(c, seed):
    if c["kind"] == "tables":
        return None
    s = prepare(c, seed)
    if c["kind"] == "rope":
        return {"q": _exact_rotated(s["q"], s["wq"], s), "k": _exact_rotated(s["k"], s["wk"], s)}
    if c["kind"] in ("fused", "append"):
        out, k = {}, s["k"]
        if c["kind"] == "fused":
            out["q"] = _exact_rotated(s["q"], s["wq"], s)
            k = _exact_rotated(k, s["wk"], s).to(k.dtype)  # the cache takes keys of the model's type
        return out | {"k": _exact_stored(k, s["slots"]), "v": _exact_stored(s["v"], s["slots"])}
    page, d, hkv, group = s["page"], c["d"], c["hkv"], c["hq"] // c["hkv"]
    outs, lses, at = [], [], 0
    for b, (n, m) in enumerate(zip(_kv_lens(c), _new_lens(c))):
        pg = s["table"][b, :-(-n // page)].long()
        code, sc = s["data"][pg].permute(2, 1, 0, 3), s["scales"][pg].permute(2, 1, 0, 4, 3)
        rows = [code[0].reshape(hkv, -1, page, d // 2),
                code[1].reshape(hkv, -1, page // 4, d // 8, 4, 4).permute(0, 1, 2, 4, 3, 5).reshape(hkv, -1, page, d // 2)]
        kv = []
        for x, y in zip(rows, sc):
            x = torch.stack([x & 15, x >> 4], dim=-1).reshape(hkv, -1, d).long()
            p, f = (x >> 1) & 3, (x & 1).double()
            val = torch.where(p > 0, (1 + f / 2) * torch.exp2((p - 1).double()), f / 2)
            val = torch.where(x >= 8, -val, val)
            sx = torch.exp2(y.reshape(hkv, -1, d // 32).double() - 127)
            kv.append((val.view(hkv, -1, d // 32, 32) * sx[..., None]).view(hkv, -1, d)[:, :n])
        q = s["q"][at:at + m].double().view(m, hkv, group, d).permute(1, 2, 0, 3).reshape(hkv, group * m, d)
        x = (q @ kv[0].transpose(1, 2) * s["scale"]).view(hkv, group, m, n)
        i, t = torch.arange(m, device="cuda")[:, None] + n - m, torch.arange(n, device="cuda")
        seen = (t <= i) & ((t > i - c["window"]) if c["window"] else torch.ones_like(t, dtype=torch.bool))
        x = torch.where(seen, x, -math.inf)
        lse = torch.logsumexp(x, -1)
        o = torch.exp(x - lse[..., None]).view(hkv, group * m, n) @ kv[1]
        outs.append(o.view(hkv, group, m, d).permute(2, 0, 1, 3).reshape(m, hkv * group, d))
        lses.append(lse.permute(2, 0, 1).reshape(m, hkv * group))
        at += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
