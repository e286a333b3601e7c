"""Cases of the serving operators: the 8-bit paged cache and the attention that reads it, sharing,
freeing and moving a cache's pages, and attention over packed prompts.

Where ``own`` is false, ``run`` computes an operator with elementary torch operations; where it is
true, it makes the calls of ``latency_collectives_amd`` that a serving program makes.

The 8-bit cache, as both sides hold it: ``data`` uint8 [pages, heads, 2, P * D] (index 0 of the third
axis is K, 1 is V) and ``scales`` uint8 [pages, heads, P / 16, 2]. K rows are plain; V rows lie by four
tokens: [P / 4][D][4]. A code is e4m3 (sign, four exponent bits, three mantissa bits, 0x7F NaN), a
scale byte s stands for 2^(s - 127) and belongs to 16 tokens of a head. A run of new tokens that
begins at a block's first token starts the block afresh; otherwise the block's scale never
falls, and where it grows the tokens already there are rounded to it.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_GOLD = 0.6180339887498949
_BLOCK = 16  # tokens of a scale


# ------------------------------------------------------------------ cases


def listed():
    return [
        # Norm, rotation and the cache's new rows of a decode step over 64 requests, one rank's heads.
        {"name": "put8_decode", "kind": "put", "dtype": "bf16", "b": 64, "new": 1, "kv": 2000, "hq": 8,
         "hkv": 1, "d": 128, "rot": 128, "inter": False, "page": 16, "fused": True},
        # Chunks of a few prompts into the cache, odd lengths, some behind tokens already there.
        {"name": "put8_prompt", "kind": "put", "dtype": "bf16", "b": 3, "new": 4001, "kv": 6007, "hq": 8,
         "hkv": 8, "d": 128, "rot": 128, "inter": False, "page": 32, "fused": False},
        # One request, one rank's heads: the smallest attention of a decode step.
        {"name": "attn8_single", "kind": "attn", "dtype": "bf16", "b": 1, "new": 1, "kv": 2000,
         "hq": 8, "hkv": 1, "d": 128, "page": 16, "window": 0},
        # An ordinary decode batch of ragged lengths.
        {"name": "attn8_decode", "kind": "attn", "dtype": "bf16", "b": 64, "new": 1, "kv": 8192,
         "hq": 32, "hkv": 8, "d": 128, "page": 16, "window": 0},
        # Chunks of prompts against what is cached already: compute-bound.
        {"name": "attn8_chunk", "kind": "attn", "dtype": "bf16", "b": 2, "new": 2048, "kv": 12288,
         "hq": 32, "hkv": 8, "d": 128, "page": 32, "window": 0},
        # One request sampled four ways on one rank, then dropped: latency counts.
        {"name": "fork_small", "kind": "fork", "b": 1, "times": 3, "kv": 1000, "page": 16, "hkv": 1,
         "d": 128, "layers": 4},
        # A batch of prompts, each sampled 16 ways, every layer's last page copied.
        {"name": "fork_large", "kind": "fork", "b": 32, "times": 16, "kv": 4096, "page": 64, "hkv": 8,
         "d": 128, "layers": 4},
        # A small pool closes its holes.
        {"name": "compact_small", "kind": "compact", "b": 8, "kv": 500, "page": 16, "hkv": 1, "d": 128,
         "layers": 2},
        # A large pool, half empty after requests left, moves its upper pages down.
        {"name": "compact_large", "kind": "compact", "b": 512, "kv": 8192, "page": 64, "hkv": 1,
         "d": 128, "layers": 2},
        # A handful of short prompts on one rank.
        {"name": "prompt_short", "kind": "prompt", "dtype": "bf16", "b": 7, "n": 301, "hq": 8, "hkv": 1,
         "d": 128, "window": 0},
        # A batch of ragged prompts over the whole layer's heads: compute-bound.
        {"name": "prompt_batch", "kind": "prompt", "dtype": "bf16", "b": 6, "n": 8191, "hq": 32, "hkv": 8,
         "d": 128, "window": 0},
        # Binary32, a small head, a sliding window, odd lengths.
        {"name": "prompt_f32_window", "kind": "prompt", "dtype": "f32", "b": 5, "n": 2049, "hq": 12,
         "hkv": 4, "d": 64, "window": 500},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    kind = rng.choice(["put", "put", "attn", "attn", "attn", "fork", "compact", "prompt", "prompt"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([64, 96, 128, 128, 192, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    if kind == "fork":
        room = 512 * 64 * 1024 * 4 // (page * hkv * d)  # pages copied over all layers
        layers = rng.choice([1, 2, 4, 8])
        most = max(1, min(512, room // layers))
        b = _log(rng, 1, min(64, most))
        return {"kind": kind, "b": b, "times": _log(rng, 1, max(1, min(32, most // b))), "page": page,
                "kv": _log(rng, 1, min(4096, 128 * page)), "hkv": hkv, "d": d, "layers": layers}
    if kind == "compact":
        layers = rng.choice([1, 2, 4])
        pages = 32768 * 64 * 128 * 2 // (page * hkv * d * layers)
        kv = _log(rng, 1, min(8192, max(1, pages * page // 16)))
        b = _log(rng, 1, max(1, min(512, pages * page // max(kv, page))))
        return {"kind": kind, "b": b, "kv": kv, "page": page, "hkv": hkv, "d": d, "layers": layers}
    if kind == "put":
        fused = rng.random() < 0.6
        new = rng.choice([1, 1, _log(rng, 2, 2000)])
        most = 8000 * 8 * 128 // (hkv * d * (2 if dtype == "f32" else 1) * (max(1, hq // hkv // 4) if fused else 1))
        b = _log(rng, 1, max(1, min(500, most // new)))
        return {"kind": kind, "dtype": dtype, "b": b, "new": new, "hq": hq, "hkv": hkv, "d": d,
                "kv": _log(rng, new, max(new, min(6000, 200000 // b))),
                "rot": rng.choice([d, d, d // 2]), "inter": rng.random() < 0.4, "page": page, "fused": fused}
    window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    if kind == "prompt":
        most = 1.5e12 if dtype == "bf16" else 1e11  # operations of all prompts
        n = _log(rng, 1, min(8191, int(math.sqrt(most / (2 * hq * d)))))
        b = _log(rng, 1, max(1, min(100, int(most / (2 * hq * d * float(n) * n)), 60000 * 128 // (n * d))))
        return {"kind": kind, "dtype": dtype, "b": b, "n": n, "hq": hq, "hkv": hkv, "d": d, "window": window}
    new = rng.choice([1, 1, 1, 2, 4, _log(rng, 8, 700)])
    kv = _log(rng, new, 65536 if new == 1 else 12000)
    most = int(4e6 if new == 1 else 6e7 / (new * hq // hkv))
    b = _log(rng, 1, max(1, min(200, most // max(1, kv * hkv))))
    return {"kind": kind, "dtype": dtype, "b": b, "new": new, "kv": kv, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "window": window}


def _ragged(most, b, shift):
    """The first has the most, others are spread over 1 .. most."""
    return [most if i == 0 else 1 + int((most - 1) * ((i * _GOLD + shift) % 1.0)) for i in range(b)]


def _new_lens(c):
    """Tokens each request brings: decode steps bring one, others 1 .. new."""
    return _ragged(c["new"], c["b"], 0.0)


def _kv_lens(c):
    """Length of each request with its new tokens."""
    return [max(n, m) for n, m in zip(_ragged(c["kv"], c["b"], 0.3), _new_lens(c))]


def _pages(lens, page):
    return sum(-(-n // page) for n in lens)


def _seen(n, m, window):
    """Places that the last m of n tokens see."""
    if not window:
        return m * (n - m) + m * (m + 1) // 2
    full = max(0, min(m, n - window))  # rows whose window is whole
    k = m - full
    return full * window + k * (n - m) + k * (k + 1) // 2


def work(c):
    es = 4 if c.get("dtype") == "f32" else 2
    if c["kind"] == "put":  # into the cache, and the touched blocks' rows read back as values
        t, rows = sum(_new_lens(c)), sum(n - (n - m) // _BLOCK * _BLOCK for n, m in zip(_kv_lens(c), _new_lens(c)))
        n = t * (2 * c["hkv"] * c["d"] * (es + 1) + 8) + rows * (2 * c["hkv"] * c["d"] * 3 + 8)
        if c["fused"]:
            n += t * (c["hq"] * c["d"] * es * 2 + c["rot"] * 4 + 4)
        return {"bytes": n, "flops": 8 * t * c["hkv"] * c["d"]}
    if c["kind"] == "attn":
        new, lens = _new_lens(c), _kv_lens(c)
        seen = sum(_seen(n, m, c["window"]) for n, m in zip(lens, new))
        read = sum(min(n, c["window"] + m - 1) if c["window"] else n for n, m in zip(lens, new))
        t = sum(new)
        return {"bytes": read * c["hkv"] * 2 * c["d"] + read * c["hkv"] * 2 // _BLOCK
                + t * c["hq"] * (2 * c["d"] * es + 4) + 4 * (_pages(lens, c["page"]) + 3 * c["b"]),
                "flops": 4 * seen * c["hq"] * c["d"]}
    if c["kind"] == "prompt":
        lens = _ragged(c["n"], c["b"], 0.3)
        seen = sum(_seen(n, n, c["window"]) for n in lens)
        t = sum(lens)
        return {"bytes": t * ((2 * c["hq"] + 2 * c["hkv"]) * c["d"] * es + 4 * c["hq"]),
                "flops": 4 * seen * c["hq"] * c["d"]}
    page_bytes = c["layers"] * c["hkv"] * 2 * c["page"] * c["d"] + c["layers"] * c["hkv"] * 2 * c["page"] // _BLOCK
    lens = _ragged(c["kv"], c["b"], 0.3)
    pages = _pages(lens, c["page"])
    if c["kind"] == "fork":
        n = c["b"] * c["times"]
        copied = sum(c["times"] for m in lens if m % c["page"])
        # rows read once and written for every fork, their pages counted up and down again
        return {"bytes": copied * page_bytes * 2 + pages * (4 + c["times"] * 20) + n * 40, "flops": 0}
    # half the live pages lie above the first `live`, in the mean
    return {"bytes": pages // 2 * page_bytes * 2 + pages * 8 + 3 * 4 * 2 * pages, "flops": 0}


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


_handles = {}


def _handle(name, *geometry):
    """What a serving program keeps for caches, or prompts, of this geometry."""
    if not own:
        return None
    import latency_collectives_amd as lc

    key = (name, *geometry)
    if key not in _handles:
        _handles[key] = getattr(lc, name)(*geometry)
    return _handles[key]


def _empty(pages, c):
    return (torch.zeros(pages, c["hkv"], 2, c["page"] * c["d"], dtype=torch.uint8, device="cuda"),
            torch.zeros(pages, c["hkv"], c["page"] // _BLOCK, 2, dtype=torch.uint8, device="cuda"))


def _filled(pages, c, g):
    """A cache of `pages` pages whose rows are normal values of different sizes."""
    stock = min(pages, 257)
    data, scales = _empty(stock, c)
    n = stock * c["page"]
    size = torch.exp(0.5 * torch.randn(2, n, c["hkv"], 1, device="cuda", generator=g))
    rows = torch.randn(2, n, c["hkv"], c["d"], device="cuda", generator=g) * size
    _put(data, scales, rows[0], rows[1], torch.arange(n, device="cuda"))
    pick = torch.randint(0, stock, (pages,), device="cuda", generator=g)
    return data[pick], scales[pick]


def _table(lens, page, pages, g, rows=None):
    """Block tables of requests of these lengths, pages in random order, and the pages left over."""
    perm = torch.randperm(pages, device="cuda", generator=g).int()
    width = max(-(-n // page) for n in lens)
    table = torch.full((rows or len(lens), width), -1, dtype=torch.int32, device="cuda")
    counts = _i32([-(-n // page) for n in lens])
    held = torch.arange(width, device="cuda")[None, :] < counts[:, None]
    n = int(counts.sum())
    table[:len(lens)][held] = perm[:n]
    return table, perm[n:]


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": c, "kind": c["kind"]}
    if c["kind"] == "prompt":
        lens, dt = _ragged(c["n"], c["b"], 0.3), _TYPES[c["dtype"]]
        t = sum(lens)
        # the projection's output: q, k and v of a token side by side
        qkv = torch.randn(t, (c["hq"] + 2 * c["hkv"]) * c["d"], device="cuda", generator=g).to(dt)
        q, k, v = (x.view(t, -1, c["d"]) for x in qkv.split([c["hq"] * c["d"], c["hkv"] * c["d"], c["hkv"] * c["d"]], dim=1))
        s.update(q=q, k=k, v=v, lens=lens, q_start=_i32(_starts(lens)), scale=1.0 / math.sqrt(c["d"]),
                 window=c["window"], handle=_handle("ar_prompt_create", c["hkv"], c["d"]),
                 out=torch.empty(t, c["hq"], c["d"], dtype=dt, device="cuda"),
                 lse=torch.empty(t, c["hq"], dtype=torch.float32, device="cuda"))
        return s
    page = c["page"]
    if c["kind"] in ("fork", "compact"):
        lens = _ragged(c["kv"], c["b"], 0.3)
        live, n = _pages(lens, page), c["b"] * c.get("times", 0)
        pages = 2 * live + 3 if c["kind"] == "compact" else live + n + 5
        rows = c["b"] + n
        table, left = _table(lens, page, pages, g, rows)
        s.update(table=table, kv_len=_i32(lens + [0] * n), page=page,
                 shares=torch.zeros(pages, dtype=torch.int32, device="cuda"),
                 scratch=torch.zeros(-(-pages // 32) + 1, dtype=torch.int32, device="cuda"),
                 pool_out=torch.zeros(2, dtype=torch.int32, device="cuda"),
                 free=torch.zeros(pages, dtype=torch.int32, device="cuda"))
        s["caches"] = [x for _ in range(c["layers"]) for x in _filled(pages, c, g)]
        if c["kind"] == "fork":
            # every request's forks side by side, into the empty rows
            s.update(src=_i32([i // c["times"] for i in range(n)]), dst=_i32([c["b"] + i for i in range(n)]),
                     pool=_i32([live, pages]), kv_forked=torch.zeros(rows, dtype=torch.int32, device="cuda"),
                     kv_freed=torch.zeros(rows, dtype=torch.int32, device="cuda"),
                     pool_freed=torch.zeros(2, dtype=torch.int32, device="cuda"),
                     copy_src=torch.zeros(n, dtype=torch.int32, device="cuda"),
                     copy_dst=torch.zeros(n, dtype=torch.int32, device="cuda"),
                     refused=torch.zeros(n, dtype=torch.int32, device="cuda"))
            s["free"][live:] = left.sort().values
            return s
        # some prefixes are held twice: a request's row begins with its neighbour's whole pages
        for b in range(1, c["b"], 5):
            whole = min(lens[b - 1], lens[b]) // page // 2
            s["table"][b, :whole] = s["table"][b - 1, :whole]
            s["shares"][s["table"][b, :whole].long()] = 1
        s.update(table_out=torch.empty_like(table), shares_out=torch.empty_like(s["shares"]),
                 move_src=torch.empty(pages // 2, dtype=torch.int32, device="cuda"),
                 move_dst=torch.empty(pages // 2, dtype=torch.int32, device="cuda"))
        return s
    dt, d, hkv = _TYPES[c["dtype"]], c["d"], c["hkv"]
    new, lens = _new_lens(c), _kv_lens(c)
    t, pages = sum(new), _pages(lens, page) + 3
    s["handle"] = _handle("ar_kv8_create", hkv, d, page)
    s["page"] = page
    s["data"], s["scales"] = _filled(pages, c, g)
    s["table"], _ = _table(lens, page, pages, g)
    if c["kind"] == "put":
        hq, pad = c["hq"], 3  # a step's buffers are padded to a fixed size
        table = s["table"].tolist()

        def slots(lo, hi):
            return [table[b][i // page] * page + i % page for b in range(c["b"]) for i in range(lo[b], hi[b])]

        had = [n - m for n, m in zip(lens, new)]
        size = torch.exp(0.5 * torch.randn(t + pad, 1, device="cuda", generator=g))
        qkv = (torch.randn(t + pad, (hq + 2 * hkv) * d, device="cuda", generator=g) * size).to(dt)
        q, k, v = (x.view(t + pad, -1, d) for x in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
        back = slots([n // _BLOCK * _BLOCK for n in had], lens)
        s.update(q=q, k=k, v=v, t=t, eps=1e-6, inter=c["inter"], had=had, lens=lens,
                 slots=torch.tensor(slots(had, lens) + [-1] * pad, dtype=torch.int64, device="cuda"),
                 back=torch.tensor(back, dtype=torch.int64, device="cuda"),
                 positions=_i32([i for b in range(c["b"]) for i in range(had[b], lens[b])] + [-1] * pad),
                 k_read=torch.empty(len(back), hkv, d, dtype=torch.bfloat16, device="cuda"),
                 v_read=torch.empty(len(back), hkv, d, dtype=torch.bfloat16, device="cuda"))
        if c["fused"]:
            s.update(cos_sin=_cos_sin(max(lens), c["rot"]),
                     q_out=torch.zeros(t + pad, hq, d, dtype=dt, device="cuda"),
                     wq=(1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(dt),
                     wk=(1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(dt))
        return s
    s.update(q=torch.randn(t, c["hq"], d, device="cuda", generator=g).to(dt), kv_len=_i32(lens),
             q_start=_i32(_starts(new)), most=max(new), scale=1.0 / math.sqrt(d), window=c["window"],
             out=torch.empty(t, c["hq"], d, dtype=dt, device="cuda"),
             lse=torch.empty(t, c["hq"], dtype=torch.float32, device="cuda"))
    return s


# ------------------------------------------------------------------ plain forms


def _codes(data, d):
    """[pages, heads, 2, P, D] codes of the cache: a copy."""
    n, heads, _, size = data.shape
    p = size // d
    k = data[:, :, 0].view(n, heads, p, d)
    v = data[:, :, 1].view(n, heads, p // 4, d, 4).transpose(3, 4).reshape(n, heads, p, d)
    return torch.stack([k, v], dim=2)


def _values(data, scales, d):
    """[pages, heads, 2, P, D] in binary32 of whole pages."""
    x = _codes(data, d).view(torch.float8_e4m3fn).float()
    size = torch.exp2(scales.float() - 127).transpose(2, 3).repeat_interleave(_BLOCK, dim=3)
    return x * size[..., None]


def _exponent(most):
    """The smallest e, -100 to 119, with most <= 448 2^e (448 = 0.875 2^9)."""
    m, e = torch.frexp(most)
    return torch.where(most > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -100)).clamp(-100, 119)


def _put(data, scales, k, v, slots):
    """Rows k, v [T, heads, D] to `slots` (negative: nowhere), the scales' rule kept for every block."""
    t, heads, d = k.shape
    pages, page = data.shape[0], data.shape[3] // d
    # a token without a slot goes to a block behind the last
    nb = pages * page // _BLOCK
    block = torch.where(slots >= 0, slots // _BLOCK, nb)
    off = torch.where(slots >= 0, slots % _BLOCK, 0)
    rows = torch.stack([k.float(), v.float()], dim=2)  # [T, heads, 2, D]
    first = torch.full((nb + 1,), _BLOCK, dtype=torch.int64, device="cuda").scatter_reduce(0, block, off, "amin")[:nb]
    each = block[:, None, None].expand(t, heads, 2)
    most = torch.zeros(nb + 1, heads, 2, device="cuda").scatter_reduce(0, each, rows.abs().amax(-1), "amax")[:nb]
    had = scales.permute(0, 2, 1, 3).reshape(nb, heads, 2).int() - 127
    e = torch.where((first < _BLOCK)[:, None, None],
                    torch.maximum(_exponent(most), torch.where((first > 0)[:, None, None], had, -100)), had)
    # every block's codes at its scale of now; those that keep theirs are unchanged
    x = _codes(data, d).view(pages, heads, 2, page // _BLOCK, _BLOCK, d).permute(0, 3, 1, 2, 4, 5).reshape(nb, heads, 2, _BLOCK, d)
    x = torch.ldexp(x.view(torch.float8_e4m3fn).float(), (had - e)[..., None, None])
    x = torch.cat([x, x.new_zeros(1, heads, 2, _BLOCK, d)])
    e_all = torch.cat([e, e.new_zeros(1, heads, 2)])
    x.permute(0, 3, 1, 2, 4)[block, off] = torch.ldexp(rows, -e_all[block][..., None])
    code = x[:nb].to(torch.float8_e4m3fn).view(torch.uint8)
    code = code.view(pages, page // _BLOCK, heads, 2, _BLOCK, d).permute(0, 2, 3, 1, 4, 5).reshape(pages, heads, 2, page, d)
    data[:, :, 0] = code[:, :, 0].reshape(pages, heads, page * d)
    data[:, :, 1] = code[:, :, 1].view(pages, heads, page // 4, 4, d).transpose(3, 4).reshape(pages, heads, page * d)
    scales.copy_((e + 127).to(torch.uint8).view(pages, page // _BLOCK, heads, 2).permute(0, 2, 1, 3))


def _norm_rope(x, w, cs, positions, eps, inter, wide):
    """Per-head RMS norm and rotation of x [T, H, D], in `wide`."""
    y = x.to(wide)
    y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * w.to(wide)
    rot = cs.shape[1]
    row = cs[positions.long()].to(wide)[:, None, :]
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])
    p, q = a * c - b * s, b * c + a * s
    p = torch.stack([p, q], dim=-1).flatten(-2) if inter else torch.cat([p, q], dim=-1)
    return torch.cat([p, y[..., rot:]], dim=-1).to(x.dtype)


def _plain_put(s):
    t, out, k = s["t"], {}, s["k"][:s["t"]]
    if s["c"]["fused"]:
        # keys go on to eight bits: 64 bits keep their roundings away from the codes' borders
        s["q_out"][:t] = _norm_rope(s["q"][:t], s["wq"], s["cos_sin"], s["positions"][:t], s["eps"], s["inter"], torch.float32)
        k = _norm_rope(k, s["wk"], s["cos_sin"], s["positions"][:t], s["eps"], s["inter"], torch.float64)
        out["q"] = s["q_out"]
    _put(s["data"], s["scales"], k, s["v"][:t], s["slots"][:t])
    x = _values(s["data"], s["scales"], k.shape[2])
    pg, off = s["back"] // s["page"], s["back"] % s["page"]
    return out | {"k": x[pg, :, 0, off].to(torch.bfloat16), "v": x[pg, :, 1, off].to(torch.bfloat16)}


def _plain_attn(s):
    page, d = s["page"], s["q"].shape[2]
    b, width = s["table"].shape
    heads = s["data"].shape[1]
    group = s["q"].shape[1] // heads
    ids = s["table"].clamp(min=0)
    x = _values(s["data"][ids].flatten(0, 1), s["scales"][ids].flatten(0, 1), d)
    # [B, heads, tokens, D]
    k, v = (x[:, :, i].reshape(b, width, heads, page, d).transpose(1, 2).reshape(b, heads, width * page, d) for i in (0, 1))
    start, lens = s["q_start"].long(), s["kv_len"].long()
    new = start[1:] - start[:-1]
    i = torch.arange(s["most"], device="cuda")
    at = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[at].view(b, s["most"], heads, group, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(b, heads, group * s["most"], d), k.transpose(2, 3).contiguous()) * s["scale"]
    x = x.view(b, heads, group, s["most"], width * page)
    t = torch.arange(width * page, device="cuda")
    pos = (lens - new)[:, None] + i  # [B, new]
    seen = (t <= pos[..., None]) & (t < lens[:, None, None])
    if s["window"]:
        seen = seen & (t > pos[..., None] - s["window"])
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, heads, group * s["most"], -1), v).view(b, heads, group, s["most"], d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(b, s["most"], heads * group, d)
    lse = (m + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(b, s["most"], heads * group)
    live = i < new[:, None]
    return {"out": o[live].to(s["q"].dtype), "lse": lse[live]}


def _plain_prompt(s):
    heads, d = s["k"].shape[1:]
    group = s["q"].shape[1] // heads
    at = 0
    for n in s["lens"]:
        q, k, v = (x[at:at + n].float().transpose(0, 1) for x in (s["q"], s["k"], s["v"]))
        i = torch.arange(n, device="cuda")
        for h in range(heads):
            x = torch.matmul(q[h * group:(h + 1) * group], k[h].t().contiguous()) * s["scale"]
            seen = i <= i[:, None]
            if s["window"]:
                seen = seen & (i > i[:, None] - s["window"])
            x = x.masked_fill_(~seen, -math.inf)
            m = x.amax(-1, keepdim=True)
            x = torch.exp_(x.sub_(m))
            total = x.sum(-1, keepdim=True)
            s["out"][at:at + n, h * group:(h + 1) * group] = (torch.matmul(x, v[h]) / total).transpose(0, 1).to(s["out"].dtype)
            s["lse"][at:at + n, h * group:(h + 1) * group] = (m + torch.log(total)).squeeze(-1).t()
        at += n
    return {"out": s["out"], "lse": s["lse"]}


def _plain_copy(caches, src, dst):
    live = (src >= 0) & (dst >= 0)
    a, b = src[live].long(), dst[live].long()
    for x in caches:
        x[b] = x[a]


def _plain_fork(s):
    page, src, dst, n = s["page"], s["src"].long(), s["dst"].long(), s["src"].numel()
    width = s["table"].shape[1]
    lens = s["kv_len"][src]
    whole, tail = lens // page, lens % page > 0
    # every destination is an empty row of its own; a fork that finds no page for its tail is refused
    at = tail.int().cumsum(0) - tail.int()
    got = ~tail | (at < s["pool"][1] - s["pool"][0])
    col = torch.arange(width, device="cuda")
    shared = (col < whole[:, None]) & got[:, None]
    rows = torch.where(shared, s["table"][src], s["table"][dst])
    s["shares"].index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    fresh = s["free"][(s["pool"][0] + at).clamp(max=s["free"].numel() - 1).long()]
    last = (col == whole[:, None]) & (tail & got)[:, None]
    tails = s["table"][src].gather(1, whole.clamp(max=width - 1).long()[:, None]).squeeze(1)
    s["table"][dst] = torch.where(last, fresh[:, None], rows)
    copied = tail & got
    s["copy_src"].copy_(torch.where(copied, tails, -1))
    s["copy_dst"].copy_(torch.where(copied, fresh, -1))
    s["refused"].copy_((~got).int())
    s["kv_forked"].copy_(s["kv_len"])
    s["kv_forked"][dst] = torch.where(got, lens, s["kv_len"][dst])
    s["pool_out"].copy_(torch.stack([s["pool"][0] + copied.sum(), s["pool"][1]]))


def _plain_free(s):
    rows = s["table"][s["dst"].long()]
    col = torch.arange(rows.shape[1], device="cuda")
    held = rows[col < (-(-s["kv_forked"][s["dst"].long()] // s["page"]))[:, None]].long()
    times = torch.zeros_like(s["shares"]).index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    freed = times > s["shares"]
    s["shares"].copy_(torch.where(freed, 0, s["shares"] - times))
    ids = torch.arange(freed.numel(), device="cuda", dtype=torch.int32)[freed]
    first = int(s["pool_out"][0])
    s["free"][first - ids.numel():first] = ids
    s["pool_freed"].copy_(torch.stack([s["pool_out"][0] - ids.numel(), s["pool_out"][1]]))
    s["kv_freed"].copy_(s["kv_forked"])
    s["kv_freed"][s["dst"].long()] = 0


def _plain_compact(s):
    page, pages = s["page"], s["shares"].numel()
    col = torch.arange(s["table"].shape[1], device="cuda")
    held = col < (-(-s["kv_len"] // page))[:, None]
    live = torch.zeros(pages, dtype=torch.bool, device="cuda")
    live[s["table"][held].long()] = True
    n = live.sum()
    ids = torch.arange(pages, device="cuda", dtype=torch.int32)
    src, dst = ids[live & (ids >= n)], ids[~live & (ids < n)]
    to = ids.clone()
    to[src.long()] = dst
    s["table_out"].copy_(torch.where(held, to[s["table"].clamp(min=0).long()], -1))
    s["move_src"].fill_(-1)
    s["move_dst"].fill_(-1)
    s["move_src"][:src.numel()] = src
    s["move_dst"][:src.numel()] = dst
    s["shares_out"].copy_(torch.where(live, s["shares"], 0))
    s["shares_out"][dst.long()] = s["shares"][src.long()]
    s["shares_out"][src.long()] = 0
    s["free"].copy_(ids)
    s["pool_out"].copy_(torch.stack([n, torch.full_like(n, pages)]))


def run(s):
    kind = s["kind"]
    lc = None
    if own:
        import latency_collectives_amd as lc
    if kind == "fork":
        if own:
            lc.ar_pages_fork(s["src"], s["dst"], s["kv_len"], s["table"], s["shares"], s["pool"], s["free"],
                             s["kv_forked"], s["pool_out"], s["copy_src"], s["copy_dst"], s["refused"], s["page"])
            lc.ar_pages_copy(s["caches"], s["copy_src"], s["copy_dst"])
            lc.ar_pages_free(s["dst"], s["kv_forked"], s["table"], s["shares"], s["pool_out"], s["free"],
                             s["kv_freed"], s["pool_freed"], s["scratch"], s["page"])
        else:
            _plain_fork(s)
            _plain_copy(s["caches"], s["copy_src"], s["copy_dst"])
            _plain_free(s)
        return {x: s[x] for x in ("table", "shares", "free", "kv_forked", "kv_freed", "pool_out", "pool_freed",
                                  "copy_src", "copy_dst", "refused", "caches")}
    if kind == "compact":
        if own:
            lc.ar_pages_compact(s["kv_len"], s["table"], s["shares"], s["table_out"], s["shares_out"], s["free"],
                                s["pool_out"], s["move_src"], s["move_dst"], s["scratch"], s["page"])
            lc.ar_pages_copy(s["caches"], s["move_src"], s["move_dst"])
        else:
            _plain_compact(s)
            _plain_copy(s["caches"], s["move_src"], s["move_dst"])
        return {x: s[x] for x in ("table_out", "shares_out", "free", "pool_out", "move_src", "move_dst", "caches")}
    if not own:
        return {"put": _plain_put, "attn": _plain_attn, "prompt": _plain_prompt}[kind](s)
    if kind == "prompt":
        lc.ar_prompt_attention(s["handle"], s["q"], s["k"], s["v"], s["q_start"], s["out"], s["lse"], s["scale"],
                               s["window"])
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "put":
        out = {}
        if s["c"]["fused"]:
            lc.ar_kv8_norm_rope_append(s["handle"], s["q"], s["k"], s["v"], s["q_out"], s["positions"], s["cos_sin"],
                                       s["slots"], s["data"], s["scales"], s["wq"], s["wk"], s["eps"], s["inter"])
            out["q"] = s["q_out"]
        else:
            lc.ar_kv8_append(s["handle"], s["k"], s["v"], s["slots"], s["data"], s["scales"])
        lc.ar_kv8_read(s["handle"], s["back"], s["data"], s["scales"], s["k_read"], s["v_read"])
        return out | {"k": s["k_read"], "v": s["v_read"]}
    lc.ar_kv8_attention(s["handle"], s["q"], s["data"], s["scales"], s["table"], s["kv_len"], s["q_start"], s["out"],
                        s["lse"], s["scale"], s["window"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ definitions in 64 bits


def _e4m3(code):
    """The values that codes stand for, from their bits."""
    x = code.long()
    p, f = (x >> 3) & 15, (x & 7).double() / 8
    y = torch.where(p > 0, (1 + f) * torch.exp2((p - 7).double()), f * 2.0 ** -6)
    y = torch.where((x & 127) == 127, math.nan, y)
    return torch.where(x >= 128, -y, y)


def _rounded(y, e):
    """y to the nearest value that a code at scale 2^e stands for."""
    a = y.abs() * torch.exp2(-e.double())
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    r = torch.round(a / step) * step  # ties to even, as the codes' last bit is
    return torch.copysign(r.clamp(max=448.0) * torch.exp2(e.double()), y)


def _scale_for(most):
    e = torch.ceil(torch.log2((most / 448).clamp(min=2.0 ** -100)))
    e = torch.where(most <= 448 * torch.exp2(e - 1), e - 1, e)  # the logarithm's rounding
    return torch.where(most > 448 * torch.exp2(e), e + 1, e).clamp(-100, 119)


def _request_rows(s, b, lo, hi):
    """K and V [2, heads, hi - lo, D] and their scales' exponents [2, heads, hi - lo] of tokens lo .. hi - 1."""
    page, d = s["page"], s["c"]["d"]
    pg = s["table"][b, lo // page:-(-hi // page)].long()
    raw, heads, n = s["data"][pg], s["data"].shape[1], pg.numel()
    k = raw[:, :, 0].reshape(n, heads, page, d)
    v = raw[:, :, 1].reshape(n, heads, page // 4, d, 4).permute(0, 1, 2, 4, 3).reshape(n, heads, page, d)
    e = s["scales"][pg].permute(3, 1, 0, 2).reshape(2, heads, -1).repeat_interleave(_BLOCK, dim=2).double() - 127
    x = torch.stack([_e4m3(y).transpose(0, 1).reshape(heads, n * page, d) for y in (k, v)])
    cut = slice(lo - lo // page * page, hi - lo // page * page)
    return (x * torch.exp2(e)[..., None])[:, :, cut], e[:, :, cut]


def _exact_rotated(x, w, s):
    y = x.double()
    y = y * torch.rsqrt((y * y).sum(2, keepdim=True) / x.shape[2] + s["eps"]) * w.double()
    rot = s["cos_sin"].shape[1]
    half = rot // 2
    cs = s["cos_sin"].double()[s["positions"][:x.shape[0]].long()]
    z = torch.complex(cs[:, :half], cs[:, half:])[:, None]
    j = torch.arange(half, device="cuda")
    a, b = (2 * j, 2 * j + 1) if s["inter"] else (j, j + half)
    turned = torch.complex(y[..., a], y[..., b]) * z
    out = y.clone()
    out[..., a], out[..., b] = turned.real, turned.imag
    return out


def _exact_put(s):
    t, out, k = s["t"], {}, s["k"][:s["t"]]
    if s["c"]["fused"]:
        out["q"] = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        out["q"][:t] = _exact_rotated(s["q"][:t], s["wq"], s)
        k = _exact_rotated(k, s["wk"], s).to(k.dtype)  # the cache takes keys of the model's type
    rows, at, parts = torch.stack([k.double(), s["v"][:t].double()]).transpose(1, 2), 0, []
    heads, d = rows.shape[1], rows.shape[3]
    for b, (had, n) in enumerate(zip(s["had"], s["lens"])):
        lo = had // _BLOCK * _BLOCK
        new = rows[:, :, at:at + n - had]
        at += n - had
        room = -(-(n - lo) // _BLOCK) * _BLOCK
        y = torch.zeros(2, heads, room, d, dtype=torch.float64, device="cuda")
        y[:, :, had - lo:n - lo] = new
        e = _scale_for(y.view(2, heads, -1, _BLOCK * d).abs().amax(-1))
        if had > lo:
            before, e0 = _request_rows(s, b, lo, had)
            y[:, :, :had - lo] = before
            e[:, :, 0] = torch.maximum(e[:, :, 0], e0[:, :, 0])
        parts.append(_rounded(y, e.repeat_interleave(_BLOCK, dim=2)[..., None])[:, :, :n - lo])
    k, v = torch.cat(parts, dim=2).transpose(1, 2)
    return out | {"k": k, "v": v}


def _exact_attention(q, k, v, scale, window):
    """q [m, Hq, D], the last m of the n tokens of k, v [heads, n, D]."""
    m, hq, d = q.shape
    heads, n = k.shape[:2]
    group = hq // heads
    x = q.double().view(m, heads, group, d).permute(1, 2, 0, 3).reshape(heads, group * m, d)
    x = (x @ k.transpose(1, 2).contiguous() * scale).view(heads, group, m, n)
    i, t = torch.arange(m, device="cuda")[:, None] + n - m, torch.arange(n, device="cuda")
    seen = (t <= i) & ((t > i - window) if window else torch.ones_like(t, dtype=torch.bool))
    x = torch.where(seen, x, -math.inf)
    lse = torch.logsumexp(x, -1)
    o = torch.exp(x - lse[..., None]).view(heads, group * m, n) @ v
    return o.view(heads, group, m, d).permute(2, 0, 1, 3).reshape(m, hq, d), lse.permute(2, 0, 1).reshape(m, hq)


def exact(c, seed):
    if c["kind"] in ("fork", "compact"):
        return None
    s = prepare(c, seed)
    if c["kind"] == "put":
        return _exact_put(s)
    outs, lses, at = [], [], 0
    if c["kind"] == "attn":
        for b, (n, m) in enumerate(zip(_kv_lens(c), _new_lens(c))):
            (k, v), _ = _request_rows(s, b, 0, n)
            o, lse = _exact_attention(s["q"][at:at + m], k, v, s["scale"], c["window"])
            outs.append(o)
            lses.append(lse)
            at += m
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    group = c["hq"] // c["hkv"]
    for n in s["lens"]:
        o = torch.empty(n, c["hq"], c["d"], dtype=torch.float64, device="cuda")
        lse = torch.empty(n, c["hq"], dtype=torch.float64, device="cuda")
        k, v = (x[at:at + n].double().transpose(0, 1) for x in (s["k"], s["v"]))
        for h in range(c["hkv"]):  # the rows of a head, a few thousand at a time
            mine = slice(h * group, (h + 1) * group)
            for r in range(0, n, 2048):
                e = min(n, r + 2048)
                o[r:e, mine], lse[r:e, mine] = _exact_attention(
                    s["q"][at + r:at + e, mine], k[h:h + 1, :e], v[h:h + 1, :e], s["scale"], c["window"])
        outs.append(o)
        lses.append(lse)
        at += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
