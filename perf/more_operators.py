"""Timed cases of a paged step over a latent cache that is held in 4 bits.

A cache row is bytes and holds one token for all heads:

    codes    latent / 2 bytes   value i is code i (e2m1) times scale i // 16; value 2 j in the low half of byte j
    key      128 bytes          64 BF16 values that serve as key only, rotated by the token's position
    scales   32 bytes           e4m3, latent / 16 of them used

Five operators, in the order of a step:

pages     gives requests the pages that their new tokens need, takes finished requests' pages back, and writes every
          token's position, cache row and valid length: what the operators behind it take.
append    norms new tokens' latents, rounds them to 4 bits, rotates their key parts and the query's.
rows      rows of the cache as BF16 (here also what append wrote).
selected  attention of every query token over its own list of cache rows (the top-k's output).
paged     attention of requests of consecutive query tokens over the first valid_len tokens of their pages.

Every function is deterministic in the case and the seed. `run` computes in plain torch (32 bits, 64 where a value may
lie next to a border of the rounding) or, with `own`, through the library.
"""
import math

import torch

own = False

PAGE = 64    # tokens per page, as in the library's configurations
ROPE = 64
BLOCK = 16   # values that share a scale
MAX_POSITIONS = 1 << 17


def listed():
    return [
        # One request's next token: nothing but latency.
        dict(name="pages 1 x 1", op="pages", requests=1, q=1, ctx=4096),
        # A busy server's step: four drafted tokens each, some requests done, some idle.
        dict(name="pages 512 x 4", op="pages", requests=512, q=4, ctx=16384),
        # One request's decode step: latency.
        dict(name="append 1 x 16 heads", op="append", tokens=1, heads=16, latent=512),
        # A long prompt's chunk with an odd token count, a head group of 16.
        dict(name="append 8191 x 16 heads", op="append", tokens=8191, heads=16, latent=512),
        # The rows of one top-2048.
        dict(name="rows 2048", op="rows", rows=2048, latent=512, cached=16384),
        # A long prefix, read back as BF16.
        dict(name="rows 131071", op="rows", rows=131071, latent=512, cached=131072),
        # One request reading a top-512: latency.
        dict(name="selected 1 x 16 x 512", op="selected", requests=1, q=1, heads=16, latent=512, k=512, ctx=16384),
        # A decode batch, one head group, top-2048, some contexts shorter than k.
        dict(name="selected 128 x 16 x 2048", op="selected", requests=128, q=1, heads=16, latent=512, k=2048,
             ctx=16384),
        # Three drafted tokens per request, an odd head count, a narrower latent, odd lists.
        dict(name="selected 21 x 3 x 20 x 1001", op="selected", requests=21, q=3, heads=20, latent=256, k=1001,
             ctx=9000),
        # A decode batch with ragged lengths, one head group: memory.
        dict(name="paged 32 x 1 x 16 x 16384", op="paged", requests=32, q=1, heads=16, latent=512, ctx=16384),
        # One long context with every head: few rows, so the length has to be split.
        dict(name="paged 1 x 1 x 128 x 131072", op="paged", requests=1, q=1, heads=128, latent=512, ctx=131072),
        # A chunk of new tokens over its context, every head, odd sizes: arithmetic, the largest.
        dict(name="paged 1 x 509 x 128 x 9000", op="paged", requests=1, q=509, heads=128, latent=512, ctx=9000),
    ]


MOST_FLOPS = 1.2e12          # of the largest listed case
MOST_SCORES = 600_000_000    # heads x tokens x keys: the plain form holds them in 32 bits


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        op = rng.choice(("pages", "append", "rows", "selected", "selected", "paged", "paged"))
        heads = rng.choice((1, 3, 8, 16, 20, 32, 40, 64, 96, 128))
        latent = rng.choice((128, 256, 384, 512, 512, 512))
        if op == "pages":
            case = dict(op=op, requests=_log(rng, 1, 1024), q=_log(rng, 1, 2048), ctx=_log(rng, 100, 131072))
            pages = -(-case["ctx"] // PAGE)
            if case["requests"] * case["q"] <= 16384 and case["requests"] * pages <= 1 << 18 and case["q"] < case["ctx"]:
                return case
            continue
        if op == "append":
            return dict(op=op, tokens=_log(rng, 1, 8191), heads=heads, latent=latent)
        if op == "rows":
            return dict(op=op, rows=_log(rng, 1, 131071), latent=latent, cached=_log(rng, 64, 131072))
        if op == "selected":
            case = dict(op=op, requests=_log(rng, 1, 128), q=_log(rng, 1, 32), heads=heads, latent=latent,
                        k=_log(rng, 17, 2048), ctx=_log(rng, 100, 16384))
        else:
            case = dict(op=op, requests=_log(rng, 1, 64), q=_log(rng, 1, 512), heads=heads, latent=latent,
                        ctx=_log(rng, 100, 131072))
        tokens = case["requests"] * case["q"]
        span = case["k"] if op == "selected" else case["ctx"]
        cached = case["requests"] * case["ctx"]
        if (work(case)["flops"] <= MOST_FLOPS and tokens * heads * span <= MOST_SCORES
                and cached <= 1 << 20 and tokens * span <= 1 << 20 and tokens <= 4096):
            return case


def row_bytes(latent):
    return latent // 2 + 2 * ROPE + 32


def _lengths(case):
    """Context length of every request: the same for every seed, spread over the upper half of the
    case's context; of several requests the last is a short one."""
    n, ctx = case["requests"], case["ctx"]
    lens = [ctx - (i * 7919) % (ctx // 2 + 1) for i in range(n)]
    if n > 1:
        short = case.get("k", 2 * case["q"])
        lens[-1] = max(1, min(ctx, short // 2))
    return lens


def _valid(case):
    """Keys each query token may see: its position in the request's context plus one (0 for a token
    before the context's start, which pads a short request)."""
    q = case["q"]
    return [max(0, n - q + 1 + j) for n in _lengths(case) for j in range(q)]


def _new_tokens(case):
    """New tokens of every request, the same for every seed: most have all of q or some, every 13th none,
    every 16th is done (-1)."""
    q = case["q"]
    return [-1 if i % 16 == 15 else 0 if i % 13 == 12 else q - (i * 5) % q for i in range(case["requests"])]


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def _cos_sin(positions):
    inv = 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float()


def _pack(values, key):
    """Rows of bytes from latent values (64 bits, [n, latent]) and rotated key parts (BF16, [n, 64])."""
    n, latent = values.shape
    v = values.unflatten(1, (latent // BLOCK, BLOCK))
    s = (v.abs().amax(2) / 6).clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(s.clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    s = (torch.round(s / step) * step).clamp(min=2.0 ** -9)     # e4m3, to the nearest even
    m = v.abs() / s[..., None]
    code = ((m > 0.25).byte() + (m >= 0.75).byte() + (m > 1.25).byte() + (m >= 1.75).byte() + (m > 2.5).byte()
            + (m >= 3.5).byte() + (m > 5).byte() + 8 * (v < 0).byte()).flatten(1)
    scales = torch.zeros(n, 32, dtype=torch.uint8, device=values.device)
    scales[:, :latent // BLOCK] = s.float().to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.cat((code[:, 0::2] | code[:, 1::2] << 4, key.contiguous().view(torch.uint8), scales), 1)


def _unpack(rows, latent):
    """Values (32 bits, [n, latent + 64]) of rows of bytes: exact."""
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=rows.device)
    code = rows[:, :latent // 2]
    code = torch.stack((code & 15, code >> 4), 2).flatten(1)
    at = latent // 2
    key = rows[:, at:at + 2 * ROPE].contiguous().view(torch.bfloat16).float()
    scale = rows[:, at + 2 * ROPE:at + 2 * ROPE + latent // BLOCK].contiguous().view(torch.float8_e4m3fn).float()
    return torch.cat((level[code.int()] * scale.repeat_interleave(BLOCK, 1), key), 1)


def _cache(g, rows, latent):
    """Rows of normed latents of unit size, already in 4 bits, and rotated key parts."""
    cache = torch.empty(rows, row_bytes(latent), dtype=torch.uint8, device="cuda")
    for i in range(0, rows, 1 << 16):
        n = min(rows - i, 1 << 16)
        cache[i:i + n] = _pack(torch.randn(n, latent, generator=g, device="cuda"), _normal(g, n, ROPE))
    return cache


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "pages":
        n, q, ctx = case["requests"], case["q"], case["ctx"]
        pages = -(-ctx // PAGE)
        new = torch.tensor(_new_tokens(case), dtype=torch.int32, device="cuda")
        most = max(1, ctx - q)
        lengths = torch.randint(most // 2, most + 1, (n,), generator=g, device="cuda").int()
        lengths[n // 2::64] = 0                                # requests that begin now (the only one does not)
        if n == 1:
            lengths[:] = most - most % PAGE                    # its next token opens a page
        owned = (lengths + PAGE - 1) // PAGE
        order = torch.randperm(n * pages, generator=g, device="cuda").int()
        table = torch.where(torch.arange(pages, device="cuda") < owned[:, None], order.view(n, pages), -1)
        left = order[(table < 0).flatten()]                    # the pages that nobody has, a stack
        free = torch.zeros_like(order)
        free[:left.numel()] = left
        # Room for most requests: where the pool is short, the last ones that need pages get none.
        room = left.numel() if n < 8 else (left.numel() if n % 2 else int((-(-new.clamp(min=0) // PAGE)).sum()) - n // 16)
        count = torch.tensor([max(0, min(room, left.numel()))], dtype=torch.int32, device="cuda")
        return dict(case=case, table=table, lengths=lengths, new=new, free=free, count=count,
                    next_lengths=torch.empty_like(lengths), next_count=torch.empty_like(count))
    latent = case["latent"]
    dim = latent + ROPE
    if case["op"] == "rows":
        n, cached = case["rows"], case["cached"]
        at = torch.randint(0, cached, (n,), generator=g, device="cuda").int()
        if n > 40:
            at[17::101] = -1                                   # empty places of a short list
        return dict(case=case, cache=_cache(g, cached, latent), rows=at)
    heads = case["heads"]
    if case["op"] == "append":
        t = case["tokens"]
        rows = -(-(t + 1) // PAGE) * PAGE
        slots = torch.randperm(rows, generator=g, device="cuda")[:t].int()
        if t >= 8:
            slots[5::97] = -1        # tokens that pad a batch have no slot
        return dict(case=case, cache=_cache(g, rows, latent), latent=_normal(g, t, latent),
                    key_rope=_normal(g, t, ROPE), query_rope=_normal(g, t, heads, ROPE),
                    query=_normal(g, t, heads, dim), every=torch.arange(rows, device="cuda").int(),
                    positions=torch.randint(0, MAX_POSITIONS, (t,), generator=g, device="cuda").int(),
                    slots=slots, cos_sin=_cos_sin(MAX_POSITIONS),
                    weight=1 + _normal(g, latent) / 8, eps=1e-6)
    n, q, ctx = case["requests"], case["q"], case["ctx"]
    pages = -(-ctx // PAGE)
    table = torch.randperm(n * pages, generator=g, device="cuda").view(n, pages).int()
    state = dict(case=case, query=_normal(g, n * q, heads, dim), cache=_cache(g, n * pages * PAGE, latent),
                 scale=192 ** -0.5)
    valid = torch.tensor(_valid(case), dtype=torch.int32, device="cuda")
    if case["op"] == "paged":
        return dict(state, valid_len=valid, block_table=table)
    # The ordered top-k of random scores: distinct positions in ascending order, short contexts whole.
    k = case["k"]
    width = max(k, ctx)
    chosen = torch.empty(n * q, k, dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda")
    for i in range(0, n * q, 1024):
        v = valid[i:i + 1024, None]
        score = torch.rand(v.shape[0], width, generator=g, device="cuda")
        score = torch.where(at < v, score, -1 - at.float())
        top = score.topk(k, dim=1).indices.int()
        chosen[i:i + 1024] = torch.where(top < v, top, width).sort(dim=1).values
    request = torch.arange(n * q, device="cuda") // q
    inside = chosen < width
    at = torch.where(inside, chosen, 0)
    physical = table[request[:, None], (at // PAGE).long()] * PAGE + at % PAGE
    return dict(state, selected=torch.where(inside, physical, -1))


def _plain_pages(s):
    q = s["case"]["q"]
    table, free, length, new = s["table"], s["free"], s["lengths"].long(), s["new"].long()
    n, pages = table.shape
    count = s["count"].long()
    done = new < 0
    add = torch.where(done, 0, new.clamp(max=q))
    add = torch.where(length + add <= pages * PAGE, add, 0)
    owned = (length + PAGE - 1) // PAGE
    need = (length + add + PAGE - 1) // PAGE - owned
    fits = (need == 0) | (need.cumsum(0) <= count)
    add, need = torch.where(fits, add, 0), torch.where(fits, need, 0)
    first = need.cumsum(0) - need - owned
    # The table's new entries, from the top of the stack downwards.
    at = torch.arange(pages, device="cuda")
    fresh = (at >= owned[:, None]) & (at < (owned + need)[:, None])
    taken = free[(count - 1 - first[:, None] - at).clamp(min=0, max=free.numel() - 1)]
    table.copy_(torch.where(fresh, taken, table))
    token = torch.arange(q, device="cuda")
    on = token < add[:, None]
    pos = length[:, None] + token
    page = table.gather(1, (pos // PAGE).clamp(max=pages - 1)).long()
    # Finished requests' pages go on top of what is left.
    back = torch.where(done, owned, 0)
    left = count - need.sum()
    to = torch.where(at < back[:, None], left + (back.cumsum(0) - back)[:, None] + at, free.numel())
    more = torch.cat((free, free[:1]))
    more.scatter_(0, to.flatten(), table.flatten())
    free.copy_(more[:-1])
    s["next_lengths"].copy_(torch.where(done, 0, length + add))
    s["next_count"].copy_(left + back.sum())
    return {"positions": torch.where(on, pos, 0).int().flatten(),
            "slots": torch.where(on, page * PAGE + pos % PAGE, -1).int().flatten(),
            "valid_len": torch.where(on, pos + 1, 0).int().flatten(), "granted": add.int(), "table": table,
            "free": free, "lengths": s["next_lengths"], "count": s["next_count"]}


def _rotate(x, cos, sin):
    a, b = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)


def _attend(query, keys, seen, scale, latent):
    """query [n, q, h, d], keys [n, c, d] or [n, q, c, d], seen [n, q, c]."""
    s = torch.einsum("nqhd,ncd->nqhc" if keys.dim() == 3 else "nqhd,nqcd->nqhc", query, keys) * scale
    s = torch.where(seen[:, :, None], s, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m.isinf(), 0.0, m))
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("nqhc,ncd->nqhd" if keys.dim() == 3 else "nqhc,nqcd->nqhd", p, keys[..., :latent])
    out = out / torch.where(total > 0, total, 1.0)
    return out.flatten(0, 1).to(torch.bfloat16), (m + total.log()).squeeze(-1).flatten(0, 1)


def _plain(s):
    case = s["case"]
    if case["op"] == "pages":
        return _plain_pages(s)
    latent, cache = case["latent"], s["cache"]
    if case["op"] == "rows":
        there = s["rows"] >= 0
        values = _unpack(cache[s["rows"].clamp(min=0).long()], latent)
        return {"rows": torch.where(there[:, None], values, 0.0).to(torch.bfloat16)}
    if case["op"] == "append":
        angle = s["cos_sin"][s["positions"].long()]
        cos, sin = angle[:, :ROPE // 2], angle[:, ROPE // 2:]
        x = s["latent"].double()      # 64 bits: a value next to a border must not change its code
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"].double()
        row = _pack(x, _rotate(s["key_rope"], cos, sin).to(torch.bfloat16))
        # Tokens without a slot write to a row behind the cache.
        more = torch.cat((cache, cache[:1]))
        more[torch.where(s["slots"] >= 0, s["slots"], cache.shape[0]).long()] = row
        cache.copy_(more[:-1])
        s["query"][..., latent:] = _rotate(s["query_rope"], cos[:, None], sin[:, None]).to(torch.bfloat16)
        return {"rows": _unpack(cache[s["every"].long()], latent).to(torch.bfloat16), "query": s["query"]}
    n, q = case["requests"], case["q"]
    query = s["query"].float().unflatten(0, (n, q))
    if case["op"] == "selected":
        seen = s["selected"] >= 0
        keys = _unpack(cache[s["selected"].clamp(min=0).long().flatten()], latent)
        out, lse = _attend(query, keys.unflatten(0, (n, q, case["k"])), seen.unflatten(0, (n, q)), s["scale"], latent)
    else:
        at = torch.arange(case["ctx"], device="cuda")
        row = s["block_table"][:, at // PAGE].long() * PAGE + at % PAGE
        seen = at < s["valid_len"].view(n, q, 1)
        keys = _unpack(cache[row.flatten()], latent).unflatten(0, (n, case["ctx"]))
        out, lse = _attend(query, keys, seen, s["scale"], latent)
    return {"out": out, "lse": lse}


def _own(s):
    import exact_bf16_top_gb300 as tk
    case = s["case"]
    if case["op"] == "pages":
        step = tk.page_step(s["table"], s["lengths"], s["new"], s["free"], s["count"], rows_per_request=case["q"],
                            page_size=PAGE, next_lengths=s["next_lengths"], next_free_count=s["next_count"])
        return {"positions": step.positions, "slots": step.slots, "valid_len": step.valid_len,
                "granted": step.granted, "table": s["table"], "free": s["free"], "lengths": s["next_lengths"],
                "count": s["next_count"]}
    latent = case["latent"]
    if case["op"] == "rows":
        return {"rows": tk.latent4_rows(s["cache"], s["rows"], latent=latent)}
    if case["op"] == "append":
        tk.latent4_append(s["cache"], s["latent"], s["key_rope"], s["positions"], s["cos_sin"], s["slots"],
                          weight=s["weight"], eps=s["eps"], query_rope=s["query_rope"], query=s["query"])
        return {"rows": tk.latent4_rows(s["cache"], s["every"], latent=latent), "query": s["query"]}
    if case["op"] == "selected":
        out, lse = tk.latent4_attend_selected(s["query"], s["cache"], s["selected"], s["scale"], latent=latent,
                                              lse=True)
    else:
        out, lse = tk.latent4_attend_paged(s["query"], s["cache"], s["valid_len"], s["block_table"], s["scale"],
                                           page_size=PAGE, rows_per_request=case["q"], latent=latent, lse=True)
    return {"out": out, "lse": lse}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    if case["op"] == "pages":
        new = _new_tokens(case)
        tokens = case["requests"] * case["q"]
        pages = -(-case["ctx"] // PAGE)
        fresh = sum(-(-v // PAGE) for v in new if v > 0)
        back = sum(pages * 3 // 4 for v in new if v < 0)
        # Lengths and new tokens, granted and next lengths; an old page each; what every token gets; pages that move.
        return {"bytes": 20 * case["requests"] + 12 * tokens + 8 * (fresh + back) + 8, "flops": 10 * tokens}
    latent = case["latent"]
    dim, held = latent + ROPE, latent // 2 + latent // BLOCK + 2 * ROPE
    if case["op"] == "rows":
        n = case["rows"]
        return {"bytes": min(n, case["cached"]) * held + n * (4 + 2 * dim), "flops": n * latent}
    heads = case["heads"]
    if case["op"] == "append":
        t = case["tokens"]
        rows = -(-(t + 1) // PAGE) * PAGE
        # New tokens read, their rows and the queries' rotated parts written, angles, ids, the weight; every row read
        # back and written as BF16.
        return {"bytes": t * (2 * dim + held + 2 * heads * ROPE * 2 + ROPE * 4 + 8) + 2 * latent
                + rows * (held + 2 * dim + 4),
                "flops": t * (8 * latent + 6 * (heads + 1) * ROPE // 2) + rows * latent}
    valid = _valid(case)
    if case["op"] == "selected":
        pairs = sum(min(v, case["k"]) for v in valid)
        lens = [min(n, case["k"] * case["q"]) for n in _lengths(case)]
        ids = len(valid) * case["k"]
    else:
        pairs = sum(valid)
        lens = _lengths(case)
        ids = len(valid) + sum(-(-n // PAGE) for n in lens)
    # Queries and every reached cache row read once, the lists or lengths and pages, outputs.
    return {"bytes": len(valid) * heads * (2 * dim + 2 * latent + 4) + sum(lens) * held + 4 * ids,
            "flops": 2 * pairs * heads * (dim + latent)}


def _held(v):
    """What 4 bits and a scale keep of values [n, latent] in 64 bits: by the nearest of the levels, written apart from
    _pack. A level's distance decides; of two at the same distance the one with an even code."""
    f64 = torch.float64
    n, latent = v.shape
    b = v.view(n, latent // BLOCK, BLOCK)
    # All e4m3 numbers from 2^-9 to 448 in order; their place is their code, from 1 on.
    grid = torch.tensor([i * 2.0 ** -9 for i in range(1, 8)]
                        + [(8 + i) / 8 * 2.0 ** e for e in range(-6, 9) for i in range(8)][:-1], dtype=f64,
                        device=v.device)
    want = (b.abs().amax(-1) / 6).contiguous()
    hi = torch.searchsorted(grid, want).clamp(1, grid.numel() - 1)
    lo = hi - 1
    d = (grid[hi] - want) - (want - grid[lo])
    up = (d < 0) | ((d == 0) & (hi % 2 == 1))        # grid[hi] has code hi + 1
    scale = grid[torch.where(up, hi, lo)]
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=f64, device=v.device)
    m = (b.abs() / scale[..., None]).clamp(max=6.0).contiguous()
    hi = torch.searchsorted(levels, m).clamp(1, 7)
    d = (levels[hi] - m) - (m - levels[hi - 1])
    up = (d < 0) | ((d == 0) & (hi % 2 == 0))
    return (torch.sign(b) * levels[torch.where(up, hi, hi - 1)] * scale[..., None]).view(n, latent)


def _read(rows, latent):
    """Rows of bytes as 64-bit values, from the format's definition: sign, exponent and fraction of either code."""
    f64 = torch.float64
    out = torch.empty(rows.shape[0], latent + ROPE, dtype=f64, device=rows.device)
    raw = rows[:, latent // 2 + 2 * ROPE:][:, :latent // BLOCK].long()
    e, f = raw >> 3 & 15, raw & 7
    scale = torch.where(e > 0, (8 + f).to(f64) * torch.exp2((e - 10).to(f64)), f.to(f64) * 2.0 ** -9)
    for half in (0, 1):
        c = (rows[:, :latent // 2].long() >> 4 * half) & 15
        e, f = c >> 1 & 3, c & 1
        v = torch.where(e > 0, (2 + f).to(f64) * torch.exp2((e - 2).to(f64)), f.to(f64) / 2)
        out[:, half:latent:2] = torch.where(c > 7, -v, v) * scale.repeat_interleave(BLOCK // 2, 1)
    raw = rows[:, latent // 2:latent // 2 + 2 * ROPE].contiguous().view(torch.bfloat16)
    out[:, latent:] = raw.to(f64)
    return out


def exact(case, seed):
    if case["op"] == "pages":
        return None
    s = prepare(case, seed)
    latent, f64 = case["latent"], torch.float64
    if case["op"] == "rows":
        out = torch.zeros(case["rows"], latent + ROPE, dtype=f64, device="cuda")
        there = torch.nonzero(s["rows"] >= 0).flatten()
        out[there] = _read(s["cache"][s["rows"][there].long()], latent)
        return {"rows": out}
    if case["op"] == "append":
        rows, query = _read(s["cache"], latent), s["query"].to(f64)
        x, w = s["latent"].to(f64), s["weight"].to(f64)
        angle = s["cos_sin"].to(f64)[s["positions"].long()]
        turn = torch.complex(angle[:, :ROPE // 2], angle[:, ROPE // 2:])

        def turned(v, by):
            pairs = torch.view_as_complex(v.to(f64).unflatten(-1, (ROPE // 2, 2)).contiguous())
            return torch.view_as_real(pairs * by).flatten(-2)

        norm = (x.pow(2).sum(-1) / latent + s["eps"]).sqrt()
        there = torch.nonzero(s["slots"] >= 0).flatten()
        at = s["slots"].long()[there]
        rows[at, :latent] = _held(x / norm[:, None] * w)[there]
        rows[at, latent:] = turned(s["key_rope"], turn)[there]
        query[:, :, latent:] = turned(s["query_rope"], turn[:, None])
        return {"rows": rows, "query": query}
    tokens, heads = s["query"].shape[:2]
    out = torch.zeros(tokens, heads, latent, dtype=f64, device="cuda")
    lse = torch.full((tokens, heads), float("-inf"), dtype=f64, device="cuda")
    values = _read(s["cache"], latent)
    for t in range(tokens):
        if case["op"] == "selected":
            rows = s["selected"][t]
            rows = rows[rows >= 0].long()
        else:
            pos = torch.arange(int(s["valid_len"][t]), device="cuda")
            pages = s["block_table"][t // case["q"]].long()
            rows = pages[pos // PAGE] * PAGE + pos % PAGE
        if rows.numel() == 0:
            continue
        keys = values[rows]
        score = (s["query"][t].to(f64) @ keys.T) * s["scale"]
        lse[t] = torch.logsumexp(score, 1)
        out[t] = torch.softmax(score, 1) @ keys[:, :latent]
    return {"out": out, "lse": lse}
