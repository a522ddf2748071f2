"""The latent-cache operators on the GPU against their formulas in 64 bits."""
from __future__ import annotations

import pytest
import torch

import exact_bf16_top_gb300 as tk
import latent_ref as R

pytestmark = pytest.mark.gpu
ROPE = 64
SCALE = 192 ** -0.5


@pytest.fixture(autouse=True)
def clean_status():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tk.load()
    tk.device_status(clear=True)
    yield
    assert tk.device_status(clear=True) == 0, "device status flags set"


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def angles(positions):
    inv = 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float()


# ------------------------------------------------------------------ append

def check_append(tokens, heads, latent, interleaved, weighted, strided, seed):
    g = gen(seed)
    dim, rows = latent + ROPE, tokens + 9
    # Strided: rows of wider tensors, as slices of a projection's output.
    cache = normal(g, rows, dim + 8)[:, :dim] if strided else normal(g, rows, dim)
    both = normal(g, tokens, latent + ROPE)
    x, key = (both[:, :latent], both[:, latent:]) if strided else (both[:, :latent].contiguous(),
                                                                  both[:, latent:].contiguous())
    if strided:
        query = normal(g, heads, tokens, dim + 16)[:, :, :dim].transpose(0, 1)
        query_rope = normal(g, tokens, heads, 3 * ROPE)[:, :, ROPE:2 * ROPE]
    else:
        query, query_rope = normal(g, tokens, heads, dim), normal(g, tokens, heads, ROPE)
    table = angles(1000)
    pos = torch.randint(0, 1000, (tokens,), generator=g, device="cuda").int()
    slots = torch.randperm(rows, generator=g, device="cuda")[:tokens].int()
    if tokens > 3:
        slots[1], slots[2] = -1, rows            # no slot
        pos[0], pos[3] = -5, 5000                # clamped
    weight = (1 + normal(g, latent) / 8) if weighted else None
    before, qbefore = cache.clone(), query.clone()
    got = tk.latent_append(cache, x, key, pos, table, slots, weight=weight, eps=1e-5, interleaved=interleaved,
                           query_rope=query_rope, query=query)
    assert got is cache
    turn = table.double()[pos.long().clamp(0, 999)]
    ref = before.double()
    tol = torch.zeros_like(ref)
    new = torch.cat((R.norm(x, weight, 1e-5) if weighted else x.double(),
                     R.rotate(key.double(), turn, interleaved)), 1)
    # One rounding to BF16 of a value computed in 32 bits: its products' errors are
    # 2^-22 of the terms, at most 2^-20 of the largest value of the row.
    bound = R.U16 * new.abs() * 1.001 + 2.0 ** -20 * new.abs().amax(1, keepdim=True)
    at = (slots >= 0) & (slots < rows)
    ref[slots[at].long()], tol[slots[at].long()] = new[at], bound[at]
    R.assert_close(cache, ref, tol, "cache")
    assert torch.equal(query[..., :latent], qbefore[..., :latent])
    qr = R.rotate(query_rope.double(), turn[:, None], interleaved)
    R.assert_close(query[..., latent:], qr, R.U16 * 1.001 * qr.abs() + 2.0 ** -20 * qr.abs().amax(-1, keepdim=True),
                   "query")


@pytest.mark.parametrize("tokens,heads,latent", [(1, 1, 128), (1, 16, 512), (2, 3, 256), (7, 5, 384),
                                                 (129, 128, 512), (1003, 20, 512)])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("strided", [False, True])
def test_append(tokens, heads, latent, interleaved, strided):
    check_append(tokens, heads, latent, interleaved, weighted=(tokens + heads) % 3 != 0, strided=strided,
                 seed=tokens * 7 + heads)


def test_append_without_queries_and_many_tokens():
    g = gen(5)
    t, latent = 40000, 128
    cache = torch.zeros(t, latent + ROPE, dtype=torch.bfloat16, device="cuda")
    x, key = normal(g, t, latent), normal(g, t, ROPE)
    slots = torch.arange(t, device="cuda", dtype=torch.int32).flip(0).contiguous()
    table = torch.cat((torch.ones(1, 32), torch.zeros(1, 32)), 1).cuda()     # no turn
    tk.latent_append(cache, x, key, torch.zeros_like(slots), table, slots)
    assert torch.equal(cache.flip(0), torch.cat((x, key), 1))


# ------------------------------------------------------------------ attention over selected rows

def selected_case(tokens, heads, latent, k, rows, seed, empty=0.1):
    g = gen(seed)
    dim = latent + ROPE
    query, cache = normal(g, tokens, heads, dim), normal(g, rows, dim)
    sel = torch.randint(0, rows, (tokens, k), generator=g, device="cuda").int()
    sel[torch.rand(tokens, k, generator=g, device="cuda") < empty] = -1
    return query, cache, sel


def check_selected(query, cache, sel, latent, scale=SCALE, **kw):
    out, lse = tk.latent_attend_selected(query, cache, sel, scale, latent=latent, lse=True, **kw)
    ref, rl, tol, tl = R.attend(query, cache, R.visible_selected(sel, cache.shape[0]), scale, latent)
    R.assert_close(out, ref, tol, "out")
    R.assert_close(lse, rl, tl, "lse")
    return out, lse


@pytest.mark.parametrize("k", [0, 1, 2, 63, 64, 65, 127, 200, 512, 1000, 2048])
def test_selected_list_lengths(k):
    check_selected(*selected_case(3, 16, 512, k, 4096, k), 512)


@pytest.mark.parametrize("heads", [1, 3, 8, 16, 17, 20, 32, 33, 40, 64, 65, 96, 128, 200, 256])
@pytest.mark.parametrize("latent", [128, 512])
def test_selected_heads(heads, latent):
    check_selected(*selected_case(5, heads, latent, 150, 1000, heads), latent)


@pytest.mark.parametrize("latent", [256, 384])
@pytest.mark.parametrize("tokens", [1, 40, 200])
def test_selected_tokens(tokens, latent):
    check_selected(*selected_case(tokens, 20, latent, 333, 5000, tokens), latent)


def test_selected_many_tokens_of_short_lists():
    check_selected(*selected_case(1500, 16, 128, 70, 3000, 9), 128)


def test_selected_empty_lists_and_empty_places():
    query, cache, sel = selected_case(6, 24, 512, 200, 1000, 1)
    sel[0] = -1                              # nothing at all
    sel[1, :150] = -1                        # whole tiles empty, then rows
    sel[2, 1:] = -1                          # one row
    sel[3, 3], sel[3, 7] = 1000, 2 ** 31 - 1   # past the cache
    sel[4, :] = 17                           # the same row every time
    sel[5, ::2] = -(2 ** 31)
    out, lse = check_selected(query, cache, sel, 512)
    assert torch.count_nonzero(out[0]).item() == 0 and torch.isneginf(lse[0]).all()


def test_selected_rows_that_nobody_sees_may_hold_anything():
    query, cache, sel = selected_case(4, 16, 512, 130, 600, 2)
    seen = torch.zeros(600, dtype=torch.bool, device="cuda")
    seen[sel[sel >= 0].long()] = True
    clean = check_selected(query, cache, sel, 512)
    cache[~seen] = float("nan")
    cache[0 if not seen[0] else int(torch.nonzero(~seen)[0])] = float("inf")
    assert all(torch.equal(a, b) for a, b in zip(clean, check_selected(query, cache, sel, 512)))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_selected_visible_nan_reaches_its_tokens_only(bad):
    query, cache, sel = selected_case(3, 16, 256, 100, 500, 3, empty=0.0)
    sel[sel == 123] = 124
    sel[1, 50] = 123
    cache[123] = bad
    query[1, :, 0] = 1.0
    out, _ = tk.latent_attend_selected(query, cache, sel, SCALE, latent=256)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[0]).all() and torch.isfinite(out[2]).all()


@pytest.mark.parametrize("scale", [0.0, 3.0, -0.5, 1e-3])
def test_selected_scales(scale):
    # 3.0: scores of hundreds, one row takes nearly all; the maximum rises many times.
    query, cache, sel = selected_case(3, 16, 512, 700, 2000, 4)
    check_selected(query, cache, sel, 512, scale=scale)


def test_selected_rising_scores():
    # Every list entry's score exceeds the last by about 4: the running maximum moves at every tile.
    query, cache, sel = selected_case(2, 16, 512, 400, 400, 5, empty=0.0)
    sel[:] = torch.arange(400, device="cuda").int()
    cache[:, 0] = torch.arange(400, device="cuda").to(torch.bfloat16)
    query[:, :, 0] = 1.0
    query[:, 8:, 0] = -1.0                   # and falls for the other heads
    check_selected(query, cache, sel, 512, scale=4.0)


def test_selected_strides_and_given_outputs():
    g = gen(6)
    latent, dim = 256, 320
    query = normal(g, 20, 5, dim + 24)[:, :, 8:8 + dim].transpose(0, 1)
    cache = normal(g, 700, dim + 40)[:, :dim]
    sel = torch.randint(-20, 700, (5, 301), generator=g, device="cuda").int()[:, 3:290]
    out = torch.empty(5, 20, latent, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(5, 20, device="cuda")
    ws = tk.latent_workspace()
    o, l = tk.latent_attend_selected(query, cache, sel, SCALE, latent=latent, out=out, lse=lse, workspace=ws)
    assert o is out and l is lse
    ref, rl, tol, tl = R.attend(query, cache, R.visible_selected(sel, 700), SCALE, latent)
    R.assert_close(out, ref, tol, "out")
    R.assert_close(lse, rl, tl, "lse")
    o, l = tk.latent_attend_selected(query, cache, sel, SCALE, latent=latent)
    assert torch.equal(o, out) and l is None
    one = tk.latent_attend_selected(query[:1], cache, sel[:1], SCALE, latent=latent)[0]
    R.assert_close(one, ref[:1], tol[:1], "one token")
    # A query broadcast over its heads.
    wide = query[:, :1].expand(5, 20, dim)
    check_selected(wide, cache, sel, latent)


def test_selected_no_tokens_and_no_cache():
    query, cache, sel = selected_case(2, 16, 512, 100, 300, 7)
    out, lse = tk.latent_attend_selected(query[:0], cache, sel[:0], SCALE, lse=True)
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16)
    out, lse = tk.latent_attend_selected(query, cache[:0], sel, SCALE, lse=True)
    assert torch.count_nonzero(out).item() == 0 and torch.isneginf(lse).all()


def test_selected_rows_past_32_bit_offsets():
    # 6.3 GB of cache: element and byte offsets of the last rows pass 2^31 and 2^32.
    rows, dim = 5_500_000, 576
    cache = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
    g = gen(8)
    cache[-300:] = normal(g, 300, dim)
    cache[:300] = normal(g, 300, dim)
    sel = torch.randint(0, 300, (2, 256), generator=g, device="cuda").int()
    sel[:, ::2] = rows - 1 - sel[:, ::2]
    check_selected(normal(g, 2, 16, dim), cache, sel, 512)


# ------------------------------------------------------------------ attention over pages

def paged_case(lens, q, heads, latent, page, seed, block_rows=None, width=None):
    """lens: context length of each request, its q new tokens the last of them."""
    g = gen(seed)
    block_rows = block_rows or page
    n, dim = len(lens), latent + ROPE
    pages = -(-max(max(lens), width or 1) // page)
    table = torch.randperm(n * pages + 3, generator=g, device="cuda")[:n * pages].view(n, pages).int()
    cache = normal(g, (n * pages + 3) * block_rows, dim)
    valid = torch.tensor([max(0, ln - q + 1 + j) for ln in lens for j in range(q)], dtype=torch.int32, device="cuda")
    return normal(g, n * q, heads, dim), cache, valid, table, dict(page_size=page, block_rows=block_rows,
                                                                   rows_per_request=q)


def check_paged(query, cache, valid, table, kw, latent, scale=SCALE):
    out, lse = tk.latent_attend_paged(query, cache, valid, table, scale, latent=latent, lse=True, **kw)
    width = kw.get("width") or table.shape[1] * kw["page_size"]
    visible = R.visible_paged(valid, table, width, kw["page_size"], kw["block_rows"], kw["rows_per_request"],
                              cache.shape[0])
    ref, rl, tol, tl = R.attend(query, cache, visible, scale, latent)
    R.assert_close(out, ref, tol, "out")
    R.assert_close(lse, rl, tl, "lse")
    return out, lse


@pytest.mark.parametrize("length", [1, 2, 63, 64, 65, 128, 129, 1000, 9000])
def test_paged_lengths(length):
    check_paged(*paged_case([length], 1, 16, 512, 64, length), 512)


@pytest.mark.parametrize("q,heads", [(1, 1), (2, 1), (3, 16), (4, 20), (5, 33), (7, 128), (70, 1), (33, 3), (2, 96),
                                     (129, 8)])
@pytest.mark.parametrize("latent", [128, 512])
def test_paged_chunks(q, heads, latent):
    check_paged(*paged_case([q + 70, max(1, q // 2), 333], q, heads, latent, 64, q * heads), latent)


@pytest.mark.parametrize("page,block_rows", [(1, 1), (2, 8), (16, 16), (16, 64), (64, 2048), (128, 128), (1024, 1024)])
def test_paged_page_sizes(page, block_rows):
    check_paged(*paged_case([300, 1, 77], 3, 16, 256, page, page, block_rows), 256)


def test_paged_ragged_batch_with_empty_rows():
    lens = [4096, 1, 64, 700, 3, 2500, 65, 129] * 3
    query, cache, valid, table, kw = paged_case(lens, 2, 16, 512, 64, 11)
    valid[8:14] = 0
    valid[20] = -7                      # clamped
    valid[21] = 2 ** 31 - 1             # clamped to the table
    out, lse = check_paged(query, cache, valid, table, kw, 512)
    assert torch.count_nonzero(out[8:14]).item() == 0 and torch.isneginf(lse[8:14]).all()


def test_paged_last_request_short_of_its_rows():
    query, cache, valid, table, kw = paged_case([200, 300, 100], 5, 16, 128, 64, 12)
    check_paged(query[:12], cache, valid[:12], table, kw, 128)


def test_paged_many_requests():
    g = torch.Generator().manual_seed(13)
    lens = torch.randint(1, 600, (700,), generator=g).tolist()
    check_paged(*paged_case(lens, 1, 8, 128, 64, 13), 128)


def test_paged_width_limits_the_table():
    query, cache, valid, table, kw = paged_case([500, 400], 1, 16, 256, 64, 14)
    table[:, 4:] = 2 ** 30              # never read: past the width
    check_paged(query, cache, valid, table, dict(kw, width=200), 256)


def test_paged_pages_outside_the_cache_are_left_out():
    query, cache, valid, table, kw = paged_case([500, 400, 64], 1, 16, 256, 64, 15)
    table[0, 2], table[0, 3], table[1, 0] = -1, 2 ** 31 - 1, 100000
    table[2, 0] = -(2 ** 31)
    out, lse = check_paged(query, cache, valid, table, kw, 256)
    assert torch.isneginf(lse[2]).all()


@pytest.mark.parametrize("heads", [1, 16, 64])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_paged_what_a_token_may_not_see_does_not_reach_it(heads, bad):
    # Stale rows past the context, and later tokens of the same chunk.
    q, latent = 6, 512
    query, cache, valid, table, kw = paged_case([100, 67], q, heads, latent, 64, 16)
    clean, _ = tk.latent_attend_paged(query, cache, valid, table, SCALE, latent=latent, **kw)
    for r, n in enumerate((100, 67)):
        i = torch.arange(n, table.shape[1] * 64, device="cuda")
        cache[table[r].long()[i // 64] * 64 + i % 64] = bad            # past the context
        cache[int(table[r, (n - 2) // 64]) * 64 + (n - 2) % 64] = bad  # the chunk's token q - 2
    query[:, :, 0] = query[:, :, 0].abs() + 0.5
    clean, _ = tk.latent_attend_paged(query, cache.nan_to_num(0.0, 0.0, 0.0), valid, table, SCALE, latent=latent, **kw)
    out, lse = tk.latent_attend_paged(query, cache, valid, table, SCALE, latent=latent, lse=True, **kw)
    for r in range(2):
        first, last = out[r * q:r * q + q - 2], out[r * q + q - 2:(r + 1) * q]
        assert torch.isfinite(first).all()
        if bad == bad and bad > 0 or bad != bad:
            assert torch.isnan(last).all()
    # The tokens before see the same as with a clean cache, up to how their rows were summed.
    ref, rl, tol, tl = R.attend(query, cache, R.visible_paged(valid, table, 128, 64, 64, q, cache.shape[0]), SCALE,
                                latent)
    for r in range(2):
        s = slice(r * q, r * q + q - 2)
        R.assert_close(out[s], ref[s], tol[s], "out")
        R.assert_close(lse[s], rl[s], tl[s], "lse")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("heads", [4, 16])
def test_paged_a_bad_query_row_stays_alone(heads, bad):
    # One (token, head) row of the chunk holds NaN or infinity: only its own output may.
    query, cache, valid, table, kw = paged_case([130, 71], 5, heads, 256, 64, 18)
    clean, cl = check_paged(query, cache, valid, table, kw, 256)
    query[1, 2] = bad
    query[8, 0, 300] = bad
    out, lse = tk.latent_attend_paged(query, cache, valid, table, SCALE, latent=256, lse=True, **kw)
    touched = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    touched[1, 2] = touched[8, 0] = True
    assert torch.equal(out[~touched], clean[~touched]) and torch.equal(lse[~touched], cl[~touched])
    assert not torch.isfinite(out[1, 2]).any()


def test_paged_rows_per_request_past_the_tokens():
    query, cache, valid, table, kw = paged_case([90], 3, 16, 128, 64, 19)
    want, _ = check_paged(query, cache, valid, table, kw, 128)
    got, _ = tk.latent_attend_paged(query, cache, valid, table, SCALE, latent=128,
                                    **dict(kw, rows_per_request=2 ** 31 - 1))
    assert torch.equal(got, want)


def test_paged_one_long_context():
    check_paged(*paged_case([50_001], 2, 16, 512, 64, 17), 512)


# ------------------------------------------------------------------ streams, repeats, the step together

def test_repeats_are_bit_equal_and_streams_are_kept():
    query, cache, sel = selected_case(9, 128, 512, 2048, 30000, 20)
    first = tk.latent_attend_selected(query, cache, sel, SCALE, lse=True)
    for _ in range(5):
        again = tk.latent_attend_selected(query, cache, sel, SCALE, lse=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [tk.latent_attend_selected(query, cache, sel, SCALE, lse=True, stream=s) for s in (side, None, side, None)]
    torch.cuda.synchronize()
    for again in got:
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_in_a_graph():
    query, cache, valid, table, kw = paged_case([3000, 100], 2, 16, 512, 64, 21)
    want = tk.latent_attend_paged(query, cache, valid, table, SCALE, lse=True, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tk.latent_attend_paged(query, cache, valid, table, SCALE, lse=True, **kw)
    valid -= 50
    graph.replay()
    later = tk.latent_attend_paged(query, cache, valid, table, SCALE, lse=True, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, later))
    assert not torch.equal(got[0], want[0])


def test_a_decode_step_append_select_attend():
    """The operators as a step uses them: append the new token, select from its scores, attend over the selection;
    a selection of everything gives what the pages give."""
    g = gen(22)
    latent, heads, n, ctx = 512, 16, 4, 1500
    dim, pages = latent + ROPE, 24
    table = torch.randperm(n * pages, generator=g, device="cuda").view(n, pages).int()
    cache = normal(g, n * pages * 64, dim)
    lens = torch.tensor([1500, 700, 1, 1024], dtype=torch.int32, device="cuda")
    last = (lens - 1).long()
    slots = (table.gather(1, (last // 64)[:, None])[:, 0] * 64 + last % 64).int()
    query = normal(g, n, heads, dim)
    tk.latent_append(cache, normal(g, n, latent), normal(g, n, ROPE), lens - 1, angles(2000), slots,
                     weight=torch.ones(latent, dtype=torch.bfloat16, device="cuda"),
                     query_rope=normal(g, n, heads, ROPE), query=query)
    logits = normal(g, n, 1536)
    for k in (256, 1536):
        rows = tk.select(logits, lens, k, tk.TOKEN, table, 64)
        out, lse = check_selected(query, cache, rows, latent)
    whole, wl = tk.latent_attend_paged(query, cache, lens, table, SCALE, lse=True)
    ref, rl, tol, tl = R.attend(query, cache, R.visible_paged(lens, table, 1536, 64, 64, 1, cache.shape[0]), SCALE,
                                latent)
    for got in (out, whole):
        R.assert_close(got, ref, tol, "out")
    for got in (lse, wl):
        R.assert_close(got, rl, tl, "lse")


# ------------------------------------------------------------------ refusals

def test_refusals():
    query, cache, sel = selected_case(2, 16, 512, 100, 300, 30)
    valid = torch.ones(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")

    def selected(q=query, c=cache, s=sel, **kw):
        return tk.latent_attend_selected(q, c, s, SCALE, **kw)

    def paged(q=query, c=cache, v=valid, t=table, **kw):
        return tk.latent_attend_paged(q, c, v, t, SCALE, **kw)

    for call in (lambda: selected(query.float()), lambda: selected(query.cpu()), lambda: selected(s=sel.long()),
                 lambda: paged(v=valid.long()), lambda: paged(c=cache.half()), lambda: paged(t=table.float())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: selected(latent=256), lambda: selected(query[..., :512]), lambda: selected(s=sel[:1]),
                 lambda: selected(c=cache[:, :512]), lambda: selected(query.transpose(1, 2)),
                 lambda: selected(out=torch.empty(2, 16, 512, device="cuda")),
                 lambda: selected(lse=torch.empty(2, 15, device="cuda")),
                 lambda: selected(workspace=torch.empty(64, device="cuda")),
                 lambda: paged(v=valid[:1]), lambda: paged(t=table[:1]), lambda: paged(page_size=48),
                 lambda: paged(width=257), lambda: paged(rows_per_request=0),
                 lambda: selected(torch.empty(1, 257, 576, dtype=torch.bfloat16, device="cuda"), s=sel[:1])):
        with pytest.raises(ValueError):
            call()
    pages = torch.zeros(2, 4000, dtype=torch.int32, device="cuda")     # long enough to need scratch
    for call, status in ((lambda: paged(t=pages, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), 1),
                         (lambda: paged(block_rows=32), 1),
                         (lambda: tk.latent_attend_selected(query, cache, sel, float("nan")), 1),
                         (lambda: selected(c=cache.flatten()[4:4 + 299 * 576].view(299, 576)), 2),
                         (lambda: selected(c=torch.empty(9, 580, dtype=torch.bfloat16, device="cuda")[:, :576]), 2)):
        with pytest.raises(tk.TopkError) as e:
            call()
        assert e.value.status == status
    x, key, pos = normal(gen(1), 2, 512), normal(gen(2), 2, ROPE), valid
    for kw in (dict(latent=x[:, :500]), dict(key_rope=key[:, :32]), dict(cos_sin=angles(4)[:, :32]),
               dict(slots=pos[:1]), dict(query=query), dict(weight=x[0, :256]), dict(cos_sin=angles(4)[:0])):
        args = dict(cache=cache, latent=x, key_rope=key, positions=pos, cos_sin=angles(4), slots=pos)
        with pytest.raises(ValueError):
            tk.latent_append(**{**args, **kw})
    with pytest.raises(TypeError):
        tk.latent_append(cache, x.float(), key, pos, angles(4), pos)


def test_the_example_decode_step():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    s = example.make(3, 5000, seed=3)
    s["lens"][1] = 700                   # fewer than k: the selection is the whole context
    s["slots"][1] = s["table"][1, 699 // 64] * 64 + 699 % 64
    out, lse, rows = example.step(s)
    ref, rl, tol, tl = R.attend(s["query"], s["cache"], R.visible_selected(rows, s["cache"].shape[0]), s["scale"], 512)
    R.assert_close(out, ref, tol, "out")
    R.assert_close(lse, rl, tl, "lse")
    assert int(s["slots"][1]) in rows[1].tolist() and (rows[1] >= 0).sum().item() == 700
    whole, wl = tk.latent_attend_paged(s["query"], s["cache"], s["lens"], s["table"], s["scale"], lse=True)
    R.assert_close(whole[1:2], ref[1:2], tol[1:2], "out of a whole context")
    assert (lse <= wl + 1e-3).all()


def test_a_scaled_down_cluster_and_shares_agree():
    # The same rows through every way of dealing the work: one token's list (a cluster), the same list for many
    # tokens (equal shares), and as pages of one token each.
    query, cache, sel = selected_case(1, 16, 256, 900, 4000, 40, empty=0.0)
    one, l1 = check_selected(query, cache, sel, 256)
    many, lm = tk.latent_attend_selected(query.expand(400, 16, 320), cache, sel.expand(400, 900).contiguous(), SCALE,
                                         latent=256, lse=True)
    paged, lp = tk.latent_attend_paged(query, cache, torch.tensor([900], dtype=torch.int32, device="cuda"), sel, SCALE,
                                       page_size=1, latent=256, lse=True)
    ref, rl, tol, tl = R.attend(query, cache, R.visible_selected(sel, 4000), SCALE, 256)
    for got, lse in ((many, lm), (paged, lp)):
        R.assert_close(got, ref.expand(got.shape), tol.expand(got.shape), "out")
        R.assert_close(lse, rl.expand(lse.shape), tl.expand(lse.shape), "lse")


@pytest.mark.parametrize("k", [128, 250, 700, 1024, 1100])
@pytest.mark.parametrize("tokens,heads", [(1, 16), (2, 128), (9, 33)])
def test_selected_short_work_in_clusters(tokens, heads, k):
    check_selected(*selected_case(tokens, heads, 384, k, 3000, k + tokens), 384)


def test_large_values_survive_a_late_maximum():
    # The largest score comes last: the weights before it are rescaled, not overflowed.
    query, cache, sel = selected_case(2, 16, 512, 300, 300, 41, empty=0.0)
    sel[:] = torch.arange(300, device="cuda").int()
    cache[:, 1:512] = (cache[:, 1:512].float() * 1e18).to(torch.bfloat16)
    query[:, :, 1:512] = 0.0
    cache[:, 0], query[:, :, 0] = 0.0, 1.0
    cache[150:, 0] = 10.0
    cache[299, 0] = 100.0
    check_selected(query, cache, sel, 512, scale=1.0)
