"""Timed cases of the latent-cache operators that stand around the top-k of a decode step.

A cache row holds one token for all heads: `latent` values that serve as key and as value, then
`rope` values that serve as key only, rotated by the token's position. Three operators:

append    norms and rotates new tokens' rows, writes them to their slots of the paged cache, and
          rotates the same tokens' query parts.
selected  attention of every query token over its own list of cache rows: the top-k's output,
          physical rows with -1 in the empty places.
paged     attention of requests of consecutive query tokens over the first valid_len tokens of
          their pages (the top-k's block table and valid lengths: one length per query token, so a
          causal chunk is lengths that grow by one).

Every function is deterministic in the case and the seed. `run` computes in plain torch (32 bits,
rounded once) or, with `own`, through the library.
"""
import torch

own = False

PAGE = 64    # tokens per page, as in the library's configurations
ROPE = 64
MAX_POSITIONS = 1 << 17


def listed():
    return [
        # One request's decode step: nothing but latency.
        dict(name="append 1 x 16 heads", op="append", tokens=1, heads=16, latent=512),
        # A decode batch of one token per request, every head on one GPU.
        dict(name="append 128 x 128 heads", op="append", tokens=128, heads=128, latent=512),
        # A long prompt's chunk with an odd token count, a head group of 16.
        dict(name="append 8191 x 16 heads", op="append", tokens=8191, heads=16, latent=512),
        # One request reading a top-512: latency.
        dict(name="selected 1 x 16 x 512", op="selected", requests=1, q=1, heads=16, latent=512, k=512, ctx=16384),
        # A decode batch, one head group, top-2048, some contexts shorter than k: memory.
        dict(name="selected 128 x 16 x 2048", op="selected", requests=128, q=1, heads=16, latent=512, k=2048,
             ctx=16384),
        # An odd batch with every head on one GPU: as much arithmetic as memory.
        dict(name="selected 37 x 128 x 2048", op="selected", requests=37, q=1, heads=128, latent=512, k=2048,
             ctx=16384),
        # Chunks of 128 new tokens of four requests, every head: arithmetic.
        dict(name="selected 512 x 128 x 2048", op="selected", requests=4, q=128, heads=128, latent=512, k=2048,
             ctx=16384),
        # One short request: latency.
        dict(name="paged 1 x 1 x 16 x 4096", op="paged", requests=1, q=1, heads=16, latent=512, ctx=4096),
        # A decode batch with ragged lengths, one head group: memory.
        dict(name="paged 32 x 1 x 16 x 16384", op="paged", requests=32, q=1, heads=16, latent=512, ctx=16384),
        # One long context with every head: few rows, so the length has to be split.
        dict(name="paged 1 x 1 x 128 x 131072", op="paged", requests=1, q=1, heads=128, latent=512, ctx=131072),
        # Four drafted tokens per request, an odd head count and a narrower latent, odd lengths.
        dict(name="paged 8 x 4 x 20 x 9000", op="paged", requests=8, q=4, heads=20, latent=256, ctx=9000),
        # A chunk of new tokens over its context, every head, odd sizes: arithmetic, the largest.
        dict(name="paged 1 x 509 x 128 x 9000", op="paged", requests=1, q=509, heads=128, latent=512, ctx=9000),
    ]


MOST_FLOPS = 1.2e12          # of the largest listed case
MOST_SCORES = 600_000_000    # heads x tokens x keys: the plain form holds them in 32 bits


def _log(rng, lo, hi):
    import math
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        op = rng.choice(("append", "selected", "selected", "paged", "paged"))
        heads = rng.choice((1, 3, 8, 16, 20, 32, 40, 64, 96, 128))
        latent = rng.choice((128, 256, 384, 512, 512, 512))
        if op == "append":
            case = dict(op=op, tokens=_log(rng, 1, 8191), heads=heads, latent=latent)
        elif op == "selected":
            case = dict(op=op, requests=_log(rng, 1, 128), q=_log(rng, 1, 32), heads=heads, latent=latent,
                        k=_log(rng, 17, 2048), ctx=_log(rng, 100, 16384))
        else:
            case = dict(op=op, requests=_log(rng, 1, 64), q=_log(rng, 1, 512), heads=heads, latent=latent,
                        ctx=_log(rng, 100, 131072))
        if op == "append":
            return case
        tokens = case["requests"] * case["q"]
        span = case["k"] if op == "selected" else case["ctx"]
        cached = case["requests"] * case["ctx"]
        if (work(case)["flops"] <= MOST_FLOPS and tokens * heads * span <= MOST_SCORES
                and cached <= 1 << 21 and tokens * span <= 1 << 21 and tokens <= 4096):
            return case


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


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def _cos_sin(positions):
    inv = 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    latent, heads, dim = case["latent"], case["heads"], case["latent"] + ROPE
    if case["op"] == "append":
        t = case["tokens"]
        rows = -(-(t + t // 4 + 1) // PAGE) * PAGE
        slots = torch.randperm(rows, generator=g, device="cuda")[:t].int()
        if t >= 8:
            slots[5::97] = -1        # tokens that pad a batch have no slot
        return dict(case=case, cache=_normal(g, rows, dim), latent=_normal(g, t, latent),
                    key_rope=_normal(g, t, ROPE), query_rope=_normal(g, t, heads, ROPE),
                    query=_normal(g, t, heads, dim),
                    positions=torch.randint(0, MAX_POSITIONS, (t,), generator=g, device="cuda").int(),
                    slots=slots, cos_sin=_cos_sin(MAX_POSITIONS),
                    weight=1 + _normal(g, latent) / 8, eps=1e-6)
    n, q, ctx = case["requests"], case["q"], case["ctx"]
    pages = -(-ctx // PAGE)
    table = torch.randperm(n * pages, generator=g, device="cuda").view(n, pages).int()
    state = dict(case=case, query=_normal(g, n * q, heads, dim), cache=_normal(g, n * pages * PAGE, dim),
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
    latent = case["latent"]
    if case["op"] == "append":
        angle = s["cos_sin"][s["positions"].long()]
        cos, sin = angle[:, :ROPE // 2], angle[:, ROPE // 2:]
        x = s["latent"].float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
        row = torch.cat((x, _rotate(s["key_rope"], cos, sin)), -1).to(torch.bfloat16)
        keep = s["slots"] >= 0
        s["cache"][s["slots"][keep].long()] = row[keep]
        s["query"][..., latent:] = _rotate(s["query_rope"], cos[:, None], sin[:, None]).to(torch.bfloat16)
        return {"cache": s["cache"], "query": s["query"]}
    n, q = case["requests"], case["q"]
    query = s["query"].float().unflatten(0, (n, q))
    if case["op"] == "selected":
        seen = s["selected"] >= 0
        keys = s["cache"][s["selected"].clamp(min=0).long()].float()
        out, lse = _attend(query, keys.unflatten(0, (n, q)), seen.unflatten(0, (n, q)), s["scale"], latent)
    else:
        at = torch.arange(case["ctx"], device="cuda")
        row = s["block_table"][:, at // PAGE].long() * PAGE + at % PAGE
        seen = at < s["valid_len"].view(n, q, 1)
        out, lse = _attend(query, s["cache"][row].float(), seen, s["scale"], latent)
    return {"out": out, "lse": lse}


def _own(s):
    import exact_bf16_top_gb300 as tk
    case = s["case"]
    if case["op"] == "append":
        tk.latent_append(s["cache"], s["latent"], s["key_rope"], s["positions"], s["cos_sin"], s["slots"],
                         weight=s["weight"], eps=s["eps"], query_rope=s["query_rope"], query=s["query"])
        return {"cache": s["cache"], "query": s["query"]}
    if case["op"] == "selected":
        out, lse = tk.latent_attend_selected(s["query"], s["cache"], s["selected"], s["scale"],
                                             latent=case["latent"], lse=True)
    else:
        out, lse = tk.latent_attend_paged(s["query"], s["cache"], s["valid_len"], s["block_table"], s["scale"],
                                          page_size=PAGE, rows_per_request=case["q"],
                                          latent=case["latent"], lse=True)
    return {"out": out, "lse": lse}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    latent, heads, dim = case["latent"], case["heads"], case["latent"] + ROPE
    if case["op"] == "append":
        t = case["tokens"]
        # New tokens read, their rows and the queries' rotated parts written, angles, ids, the weight.
        return {"bytes": t * (2 * dim * 2 + 2 * heads * ROPE * 2 + ROPE * 4 + 8) + 2 * latent,
                "flops": t * (4 * latent + 6 * (heads + 1) * ROPE // 2)}
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
    return {"bytes": len(valid) * heads * (2 * dim + 2 * latent + 4) + sum(lens) * 2 * dim + 4 * ids,
            "flops": 2 * pairs * heads * (dim + latent)}


def exact(case, seed):
    s = prepare(case, seed)
    latent, f64 = case["latent"], torch.float64
    if case["op"] == "append":
        cache, query = s["cache"].to(f64), s["query"].to(f64)
        x, w = s["latent"].to(f64), s["weight"].to(f64)
        angle = s["cos_sin"].to(f64)[s["positions"].long()]
        turn = torch.complex(angle[:, :ROPE // 2], angle[:, ROPE // 2:])

        def turned(v, by):
            pairs = torch.view_as_complex(v.to(f64).unflatten(-1, (ROPE // 2, 2)).contiguous())
            return torch.view_as_real(pairs * by).flatten(-2)

        norm = (x.pow(2).sum(-1) / latent + s["eps"]).sqrt()
        key = turned(s["key_rope"], turn)
        there = torch.nonzero(s["slots"] >= 0).flatten()
        at = s["slots"].long()[there]
        cache[at, :latent] = (x / norm[:, None] * w)[there]
        cache[at, latent:] = key[there]
        query[:, :, latent:] = turned(s["query_rope"], turn[:, None])
        return {"cache": cache, "query": query}
    tokens, heads = s["query"].shape[:2]
    out = torch.zeros(tokens, heads, latent, dtype=f64, device="cuda")
    lse = torch.full((tokens, heads), float("-inf"), dtype=f64, device="cuda")
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
        keys = s["cache"][rows].to(f64)
        score = (s["query"][t].to(f64) @ keys.T) * s["scale"]
        lse[t] = torch.logsumexp(score, 1)
        out[t] = torch.softmax(score, 1) @ keys[:, :latent]
    return {"out": out, "lse": lse}
