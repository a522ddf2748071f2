"""The latent-cache operators on the GPU at the edges of their inputs: scores of
-inf, ways of dealing the work, layouts of pages, and what is refused."""
from __future__ import annotations

import pytest
import torch

import exact_bf16_top_gb300 as tk
import latent_ref as R
from exact_bf16_top_gb300._latent_abi import Attend
from test_latent_gpu import (ROPE, SCALE, angles, check_paged, check_selected, clean_status, gen, normal,  # noqa: F401
                             paged_case, selected_case)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ scores of -inf

def listed_or_paged(form, tokens, heads, latent, length, seed):
    """One cache row per token in a shuffled order, every query token over all `length` of them: the
    rows' order [length], and a call of either form."""
    query, cache, _ = selected_case(tokens, heads, latent, 1, -(-length // 64) * 64, seed)
    if form == "listed":
        order = torch.randperm(length, generator=gen(seed), device="cuda").int()
        lists = order.expand(tokens, length).contiguous()

        def call(q, c):
            return tk.latent_attend_selected(q, c, lists, SCALE, latent=latent, lse=True)
    else:
        pages = cache.shape[0] // 64
        table = torch.randperm(pages, generator=gen(seed), device="cuda").int()
        at = torch.arange(length, device="cuda")
        order = table[at // 64] * 64 + (at % 64).int()
        valid = torch.full((tokens,), length, dtype=torch.int32, device="cuda")

        def call(q, c):
            return tk.latent_attend_paged(q, c, valid, table[None], SCALE, latent=latent, lse=True,
                                          rows_per_request=tokens)
    return query, cache, order.long(), call


# 1 token of 2048 rows is dealt to a cluster, of 30000 rows in shares of a few blocks; 200 listed tokens (tiles) of
# 700 rows in shares of many.
@pytest.mark.parametrize("form,tokens,length", [("listed", 1, 2048), ("listed", 1, 30000), ("listed", 200, 700),
                                                ("paged", 1, 2048), ("paged", 1, 30000), ("paged", 3, 700)])
@pytest.mark.parametrize("first,blocks", [(0, 1), (0, 2), (0, 5), (3, 7), (0, 10 ** 6)])
@pytest.mark.parametrize("how", ["rotary", "overflow"])
def test_scores_of_minus_infinity_weigh_nothing(form, tokens, length, first, blocks, how):
    heads, latent = 16, 256
    query, cache, order, call = listed_or_paged(form, tokens, heads, latent, length, 50)
    gone = torch.zeros(length, dtype=torch.bool, device="cuda")
    gone[first * 64:(first + blocks) * 64] = True
    query[..., latent] = 1.0 if how == "rotary" else 2.0 ** 127
    cache[:, latent] = 0.0
    cache[order[gone], latent] = float("-inf") if how == "rotary" else -(2.0 ** 127)
    out, lse = call(query, cache)
    if gone.all():
        assert torch.count_nonzero(out).item() == 0 and torch.isneginf(lse).all()
        return
    query[..., latent] = 0.0
    ref, rl, tol, tl = R.attend(query, cache, [order[~gone]] * tokens, SCALE, latent)
    R.assert_close(out, ref, tol, "out")
    R.assert_close(lse, rl, tl, "lse")


@pytest.mark.parametrize("heads", [4, 16])
@pytest.mark.parametrize("blocks", [1, 3])
@pytest.mark.parametrize("scale", [SCALE, -SCALE])
def test_a_score_of_minus_infinity_masks_whatever_its_row_holds(heads, blocks, scale):
    # A row whose latent part holds an infinity, at -inf for half of the heads (which give what they give without it)
    # and at +inf for the others: in a block that all rows see whole, in one that they do not, and at a place that only
    # the chunk's later tokens see.
    q, latent = 3, 256
    n = 64 * blocks
    query, cache, valid, table, kw = paged_case([n, n], q, heads, latent, 64, 51)
    row = table.long()[:, :, None] * 64 + torch.arange(64, device="cuda")
    row = row.flatten(1)
    low = heads // 2
    query[:, :low, 3], query[:, low:, 3] = 1.0, -1.0
    early = 10 if blocks == 1 else 74
    for r, at in ((0, early), (1, n - 2)):
        cache[row[r, at], 3] = float("-inf") * scale
        cache[row[r, at], 200] = 5.0
    out, lse = tk.latent_attend_paged(query, cache, valid, table, scale, latent=latent, lse=True, **kw)
    visible = R.visible_paged(valid, table, n, 64, 64, q, cache.shape[0])
    clean, sees = cache.clone(), []
    for t, rows in enumerate(visible):
        bad = row[t // q, early if t // q == 0 else n - 2]
        sees.append(bool((rows == bad).any()))
        visible[t] = rows[rows != bad]
        clean[bad, 3] = 0.0
    assert sees == [True] * q + [False, True, True]
    ref, rl, tol, tl = R.attend(query, clean, visible, scale, latent)
    for t in range(2 * q):
        R.assert_close(out[t, :low], ref[t, :low], tol[t, :low], f"out of token {t}")
        R.assert_close(lse[t, :low], rl[t, :low], tl[t, :low], f"lse of token {t}")
        if sees[t]:
            assert torch.isnan(out[t, low:]).all()
        else:
            R.assert_close(out[t, low:], ref[t, low:], tol[t, low:], f"out of token {t}")


def test_a_listed_score_of_minus_infinity_masks_whatever_its_row_holds():
    query, cache, sel = selected_case(3, 16, 512, 200, 1000, 52)
    query[:, :, 0] = 1.0
    sel[sel == 999] = -1
    rest = sel.clone()
    for t, i in ((0, 199), (1, 20), (2, 100)):
        sel[t, i], rest[t, i] = 999, -1
    ref, rl, tol, tl = R.attend(query, cache, R.visible_selected(rest, 1000), SCALE, 512)
    cache[999, 0] = float("-inf")
    out, lse = tk.latent_attend_selected(query, cache, sel, SCALE, lse=True)
    R.assert_close(out, ref, tol, "out")
    R.assert_close(lse, rl, tl, "lse")
    # Lists without empty places: whole blocks.
    sel = torch.randint(0, 999, (3, 192), generator=gen(53), device="cuda").int()
    rest = sel.clone()
    for t, i in ((0, 5), (1, 70), (2, 191)):
        sel[t, i], rest[t, i] = 999, -1
    cache[999, 0] = 0.0
    ref, rl, tol, tl = R.attend(query, cache, R.visible_selected(rest, 1000), SCALE, 512)
    cache[999, 0] = float("-inf")
    out, lse = tk.latent_attend_selected(query, cache, sel, SCALE, lse=True)
    R.assert_close(out, ref, tol, "out")
    R.assert_close(lse, rl, tl, "lse")


# ------------------------------------------------------------------ arguments

def test_counts_past_31_bits_are_refused():
    query, cache, valid, table, kw = paged_case([100], 1, 16, 128, 64, 60)
    for rows in (2 ** 31, 2 ** 32 + 64, 64 - 2 ** 32):
        with pytest.raises(ValueError):
            tk.latent_attend_paged(query, cache, valid, table, SCALE, latent=128, block_rows=rows)
    lists = torch.empty((1, 2 ** 32 + 100), dtype=torch.int32, device="cuda")      # 17 GB, never read
    lists[:, :100] = -1
    try:
        with pytest.raises(ValueError):
            tk.latent_attend_selected(query, cache, lists, SCALE, latent=128)
    finally:
        del lists
        torch.cuda.empty_cache()


class OtherStream:
    """Stands for a stream of another device (a test machine has one)."""
    device = torch.device("cuda", 1)
    device_index = 1
    cuda_stream = 0


def test_a_stream_of_another_device_is_refused():
    query, cache, sel = selected_case(2, 16, 512, 100, 300, 61)
    valid = torch.ones(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    x, key = normal(gen(1), 2, 512), normal(gen(2), 2, ROPE)
    slots = torch.arange(2, device="cuda", dtype=torch.int32)
    for call in (lambda s: tk.latent_attend_selected(query, cache, sel, SCALE, stream=s),
                 lambda s: tk.latent_attend_paged(query, cache, valid, table, SCALE, stream=s),
                 lambda s: tk.latent_append(cache, x, key, valid, angles(4), slots, stream=s)):
        with pytest.raises(ValueError):
            call(OtherStream())
    assert torch.cuda.current_device() == 0


def test_what_wants_a_gradient_is_refused():
    query, cache, sel = selected_case(2, 16, 512, 100, 300, 62)
    valid = torch.ones(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    x, key = normal(gen(1), 2, 512), normal(gen(2), 2, ROPE)
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    args = dict(cache=cache, latent=x, key_rope=key, positions=valid, cos_sin=angles(4),
                slots=torch.tensor([3, 4], dtype=torch.int32, device="cuda"), weight=w,
                query_rope=normal(gen(3), 2, 16, ROPE), query=query)

    want = {n: t.clone().requires_grad_() for n, t in args.items() if t.is_floating_point()}
    assert len(want) == 7
    calls = [lambda: tk.latent_attend_selected(want["query"], cache, sel, SCALE),
             lambda: tk.latent_attend_selected(query, want["cache"], sel, SCALE),
             lambda: tk.latent_attend_paged(want["query"], cache, valid, table, SCALE),
             lambda: tk.latent_attend_paged(query, want["cache"], valid, table, SCALE)]
    calls += [lambda n=n: tk.latent_append(**{**args, n: want[n]}) for n in want]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
        for mode in (torch.no_grad(), torch.inference_mode()):
            with mode:
                call()


def test_lse_by_any_truth_value():
    query, cache, sel = selected_case(2, 16, 128, 100, 300, 63)
    out, want = check_selected(query, cache, sel, 128)
    for yes in (True, 1, torch.ones(1).bool().numpy()[0]):
        assert torch.equal(tk.latent_attend_selected(query, cache, sel, SCALE, latent=128, lse=yes)[1], want)
    for no in (False, None, 0):
        assert tk.latent_attend_selected(query, cache, sel, SCALE, latent=128, lse=no)[1] is None


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("tokens,heads", [(1, 3), (5, 16), (700, 33)])
def test_append_rotates_queries_in_place(interleaved, tokens, heads):
    g, latent = gen(64), 128
    query = normal(g, tokens, heads, latent + ROPE)
    x, key, table = normal(g, tokens, latent), normal(g, tokens, ROPE), angles(900)
    slots = torch.arange(tokens, device="cuda", dtype=torch.int32)
    caches = [torch.zeros(tokens, latent + ROPE, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    apart, together = query.clone(), query.clone()
    tk.latent_append(caches[0], x, key, slots, table, slots, interleaved=interleaved,
                     query_rope=query[..., latent:].clone(), query=apart)
    tk.latent_append(caches[1], x, key, slots, table, slots, interleaved=interleaved,
                     query_rope=together[..., latent:], query=together)
    assert torch.equal(apart, together) and torch.equal(*caches)


# ------------------------------------------------------------------ the dealing of work

@pytest.mark.parametrize("short_of_sms", [0, 1, 8])
def test_ragged_pages_are_dealt_in_shares(short_of_sms):
    # As many tiles as SMs, one of them long: lengths are on the device, so the table's width must not keep a tile
    # to one CTA. Shares need scratch, whole tiles do not.
    n = torch.cuda.get_device_properties(0).multi_processor_count - short_of_sms
    lib = tk.load()
    for width in (2048, 16384, 131072):
        args = Attend(query=4096, query_token_stride=16 * 192, query_head_stride=192, cache=4096, cache_stride=192,
                      valid_len=4096, block_table=4096, out=4096, cache_rows=64, tokens=n, heads=16, latent=128,
                      width=width, table_stride=width // 64, page_size=64, block_rows=64, rows_per_request=1,
                      scale=0.1)
        assert lib.latent_bf16_attend_workspace(args, 1) > 0, width
    lens = [20000] + [70 + i for i in range(n - 1)]
    check_paged(*paged_case(lens, 1, 16, 128, 64, 70), 128)


@pytest.mark.parametrize("lens", [[1500] * 140, [1500 - 9 * i for i in range(60)] + [1500] * 80, [1500] * 100 + [1] * 40,
                                  [2000 + i for i in range(152)]])
@pytest.mark.parametrize("heads", [16, 64])
def test_pages_of_about_as_many_tiles_as_sms(lens, heads):
    query, cache, valid, table, kw = paged_case(lens, 1, heads, 128, 64, 76)
    valid[7] = 0
    check_paged(query, cache, valid, table, kw, 128)


def test_a_long_tile_among_many_short_ones():
    # Rows enough for a warp per row in the joining kernel, and a tile of more parts than a warp has lanes.
    check_paged(*paged_case([40000] + [500] * 99, 1, 16, 256, 64, 71), 256)
    check_paged(*paged_case([300] * 60 + [30001] + [77] * 30, 1, 64, 128, 64, 72), 128)


def test_many_tiles_of_64_rows_of_the_widest_latent():
    # More tiles than SMs: several pieces a CTA, tiles split between CTAs, a last tile of few rows.
    check_selected(*selected_case(230, 70, 512, 333, 3000, 73), 512)
    lens = [200 + (i * 37) % 190 for i in range(90)]
    query, cache, valid, table, kw = paged_case(lens, 3, 67, 512, 64, 74)
    check_paged(query[:268], cache, valid[:268], table, kw, 512)


def test_whole_tiles_of_ragged_listed_rows():
    # About as many tokens as SMs, each its own tile, lists between empty and full.
    query, cache, sel = selected_case(128, 16, 512, 640, 5000, 75)
    for t in range(128):
        sel[t, (t * 53) % 641:] = -1
    check_selected(query, cache, sel, 512)


# ------------------------------------------------------------------ layouts of pages

def test_paged_strided_cache_and_given_outputs():
    query, cache, valid, table, kw = paged_case([333, 200, 64], 4, 20, 256, 64, 80)
    want, wl = check_paged(query, cache, valid, table, kw, 256)
    wide = normal(gen(81), cache.shape[0], 320 + 40)[:, :320]
    wide.copy_(cache)
    q = normal(gen(82), 20, 12, 320 + 24)[:, :, 8:328].transpose(0, 1)
    q.copy_(query)
    t = torch.full((3, table.shape[1] + 5), 2 ** 30, dtype=torch.int32, device="cuda")[:, 2:2 + table.shape[1]]
    t.copy_(table)
    out = torch.empty(12, 20, 256, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(12, 20, device="cuda")
    got = tk.latent_attend_paged(q, wide, valid, t, SCALE, latent=256, out=out, lse=lse,
                                 workspace=tk.latent_workspace(), **kw)
    assert got[0] is out and got[1] is lse
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("rows", [150, 190, 63, 65])
def test_paged_last_page_ends_with_the_cache(rows):
    # Pages lead past the cache's last row in their middle: those tokens are left out.
    query, cache, valid, table, kw = paged_case([256, 100], 2, 16, 256, 64, 83)
    table[0], table[1] = torch.tensor([2, 0, 1, 3]), torch.tensor([1, 2, 0, 3])
    check_paged(query, cache[:rows], valid, table, kw, 256)


def test_paged_rows_past_32_bit_offsets():
    pages, dim = 86_000, 576                    # 6.3 GB of cache
    cache = torch.empty(pages * 64, dim, dtype=torch.bfloat16, device="cuda")
    g = gen(84)
    cache[-640:], cache[:640] = normal(g, 640, dim), normal(g, 640, dim)
    table = torch.tensor([[pages - 1, 3, pages - 7, 0, pages - 10], [1, pages - 2, 9, pages - 3, 5]],
                         dtype=torch.int32, device="cuda")
    valid = torch.tensor([317, 318, 200, 201], dtype=torch.int32, device="cuda")
    check_paged(normal(g, 4, 16, dim), cache, valid, table,
                dict(page_size=64, block_rows=64, rows_per_request=2), 512)


# ------------------------------------------------------------------ the size of the errors

@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("length", [100, 2048])
def test_errors_are_of_two_roundings(heads, length):
    # Of independent values of zero mean the weights' rounding (relative, at most 2^-8, so at most 2^-8 / sqrt 3 in the
    # mean square) leaves the same share of the output's mean square, and the output's own rounding as much again:
    # together sqrt(2 / 3) 2^-8 = 0.0032, with a tenth for the sample.
    query, cache, sel = selected_case(40, heads, 512, length, 9000, 90)
    out, _ = tk.latent_attend_selected(query, cache, sel, SCALE)
    ref = R.attend(query, cache, R.visible_selected(sel, 9000), SCALE, 512)[0]
    assert ((out.double() - ref).pow(2).mean() / ref.pow(2).mean()).sqrt().item() < 1.1 * (2 / 3) ** 0.5 * 2.0 ** -8
    query, cache, valid, table, kw = paged_case([length, length // 2], 20, heads, 512, 64, 91)
    out, _ = tk.latent_attend_paged(query, cache, valid, table, SCALE, **kw)
    ref = R.attend(query, cache, R.visible_paged(valid, table, table.shape[1] * 64, 64, 64, 20, cache.shape[0]), SCALE,
                   512)[0]
    assert ((out.double() - ref).pow(2).mean() / ref.pow(2).mean()).sqrt().item() < 1.1 * (2 / 3) ** 0.5 * 2.0 ** -8
