"""The 4-bit latent cache's operators on the GPU against their formulas in 64 bits."""
from __future__ import annotations

import pytest
import torch

import exact_bf16_top_gb300 as tk
import latent4_ref as Q
import latent_ref as R
from test_latent_gpu import ROPE, SCALE, angles, clean_status, gen, normal  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append and rows

def check_append(x, weight, eps, seed, interleaved=True, heads=3, strided=False):
    """Appends x's rows at shuffled slots (two without) and looks at every byte of the cache."""
    g = gen(seed)
    tokens, latent = x.shape
    dim, rows = latent + ROPE, tokens + 9
    cache = Q.random_cache(g, rows, latent, pad=64 if strided else 0)
    key = normal(g, tokens, ROPE)
    if strided:
        x, key = torch.cat((x, key), 1)[:, :latent], torch.cat((x, key), 1)[:, latent:]
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
    before, qbefore = cache.clone(), query.clone()
    got = tk.latent4_append(cache, x, key, pos, table, slots, weight=weight, eps=eps, interleaved=interleaved,
                            query_rope=query_rope, query=query)
    assert got is cache
    v = x.double()
    if weight is not None:
        v = R.norm(x, weight, eps)
    code, scale = Q.quantise(v)
    at = (slots >= 0) & (slots < rows)
    to = slots[at].long()
    half, used = latent // 2, latent // 16
    # Codes are those of exact arithmetic, so they are equal; a zero's sign is free.
    want = torch.where((v < 0) & (code > 0), code + 8, code)[at]
    held = torch.stack((cache[to, :half].long() & 15, cache[to, :half].long() >> 4), 2).flatten(1)
    held = torch.where(held == 8, 0, held)
    fine = (scale[at] != 0x7F).repeat_interleave(16, 1)     # (not finite: any codes)
    assert torch.equal(cache[to, half + 2 * ROPE:half + 2 * ROPE + used].long(), scale[at])
    assert torch.equal(held[fine], want[fine])
    turn = table.double()[pos.long().clamp(0, 999)]
    new = R.rotate(key.double(), turn, interleaved)
    bound = R.U16 * new.abs() * 1.001 + 2.0 ** -20 * new.abs().amax(1, keepdim=True)
    R.assert_close(Q.unpack(cache, latent)[to, latent:], new[at], bound[at], "key part")
    # Nothing else is written: other rows, unused scales.
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[to] = False
    assert torch.equal(cache[rest], before[rest])
    assert torch.equal(cache[:, half + 2 * ROPE + used:], before[:, half + 2 * ROPE + used:])
    assert torch.equal(query[..., :latent], qbefore[..., :latent])
    qr = R.rotate(query_rope.double(), turn[:, None], interleaved)
    R.assert_close(query[..., latent:], qr, R.U16 * 1.001 * qr.abs() + 2.0 ** -20 * qr.abs().amax(-1, keepdim=True),
                   "query")


@pytest.mark.parametrize("tokens,heads,latent", [(1, 1, 128), (1, 16, 512), (2, 3, 256), (7, 5, 384),
                                                 (129, 128, 512), (1003, 20, 512), (5000, 1, 256)])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("strided", [False, True])
def test_append(tokens, heads, latent, interleaved, strided):
    g = gen(tokens + heads)
    weight = (1 + normal(g, latent) / 8) if (tokens + heads) % 3 else None
    check_append(normal(g, tokens, latent), weight, 1e-5, tokens * 7 + heads, interleaved, heads, strided)


def test_append_values_on_the_borders():
    # Without a norm: every BF16 value that is a border between two codes, for scales of every size, and the largest
    # values that are borders between two scales.
    latent = 512
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], device="cuda")
    grid = Q.e4m3(torch.arange(1, 0x7F, device="cuda"))
    x = torch.zeros(4 * 126, latent, device="cuda", dtype=torch.float64)
    for sign in (0, 1):
        for i in range(126):
            s = grid[i]
            x[2 * i + sign, :8] = border * s * (-1) ** sign
            x[2 * i + sign, 16:24] = border.flip(0) * s
            if i < 125:
                x[252 + 2 * i + sign, :] = (s + grid[i + 1]) / 2 * 6 * (1 if sign else 1 - 2.0 ** -8)
    check_append(x.to(torch.bfloat16), None, 1e-6, 1)


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -12, 1e-3, 30.0, 1e4, 2.0 ** 50])
@pytest.mark.parametrize("weighted", [True, False])
def test_append_sizes(size, weighted):
    g = gen(3)
    x = (normal(g, 200, 256).float() * size).to(torch.bfloat16)
    x[5] = 0
    x[6, 1:] = 0
    weight = (normal(g, 256).float() * 3).to(torch.bfloat16) if weighted else None
    check_append(x, weight, 1e-6, 4)
    check_append(x, weight, 0.125, 4)


def test_append_norms_next_to_borders():
    # Rows of equal sizes whose norm is exactly one or nearly so: with eps = 0, x / sqrt(mean(x^2)) is +-1 and the
    # quotient by the scale 6 / 32 lands on the grid's numbers; with eps beside it by one part in 2^20 or so.
    g = gen(6)
    x = torch.where(torch.rand(300, 512, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    x = (x * torch.exp2(torch.randint(-8, 8, (300, 1), generator=g, device="cuda").float())).to(torch.bfloat16)
    weight = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 64, device="cuda").to(torch.bfloat16)
    for eps in (0.0, 2.0 ** -30, 2.0 ** -20, 1e-6):
        check_append(x, weight, eps, 7)


def test_append_not_finite():
    g = gen(8)
    x = normal(g, 12, 512)
    x[4, 17], x[5, 40], x[6, 500] = float("nan"), float("inf"), float("-inf")
    check_append(x, None, 1e-6, 9)
    cache = torch.zeros(12, 416, dtype=torch.uint8, device="cuda")
    slots = torch.arange(12, device="cuda", dtype=torch.int32)
    tk.latent4_append(cache, x, normal(g, 12, ROPE), slots, angles(20), slots,
                      weight=torch.ones(512, dtype=torch.bfloat16, device="cuda"))
    got = tk.latent4_rows(cache, slots)[:, :512]
    assert torch.isnan(got[4:7]).all() and torch.isfinite(got[:4]).all() and torch.isfinite(got[7:]).all()
    # A sum of squares past 2^127 reads as NaN, a row of zeros without eps too.
    big = torch.full((2, 512), 2.0 ** 63, device="cuda").to(torch.bfloat16)
    big[1] = 0
    tk.latent4_append(cache, big, normal(g, 2, ROPE), slots[:2], angles(20), slots[:2], eps=0.0,
                      weight=torch.ones(512, dtype=torch.bfloat16, device="cuda"))
    assert torch.isnan(tk.latent4_rows(cache, slots[:2])[:, :512]).all()


def test_append_keeps_the_sign_of_zeros():
    # -0 and what rounds to it have code 8, +0 and what rounds to it code 0, whatever the scale.
    x = torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda")
    x[0, ::2] = -0.0
    x[1] = torch.tensor([-0.0, 0.0, -0.125, 0.125, 6, -6, 1, -1] * 16)
    x[2] = torch.tensor([-0.0, 0.0, 2.0 ** -133, -(2.0 ** -133), 1.5 * 2.0 ** 60, 0.0, 0.0, -0.0] * 16)
    slots = torch.arange(3, device="cuda", dtype=torch.int32)
    for weight in (None, torch.ones(128, dtype=torch.bfloat16, device="cuda")):
        cache = torch.zeros(3, 224, dtype=torch.uint8, device="cuda")
        tk.latent4_append(cache, x, torch.zeros(3, ROPE, dtype=torch.bfloat16, device="cuda"), slots, angles(4), slots,
                          weight=weight, eps=1.0)
        code = torch.stack((cache[:, :64] & 15, cache[:, :64] >> 4), -1).flatten(1)
        small = x.abs() <= 0.125
        assert torch.equal(code[small] & 7, torch.zeros_like(code[small]))
        assert torch.equal(code >> 3 == 1, torch.signbit(x.float()))


@pytest.mark.parametrize("interleaved", [True, False])
def test_append_rotates_queries_in_place_and_works_without_them(interleaved):
    g, latent, tokens, heads = gen(64), 128, 50, 20
    query = normal(g, tokens, heads, latent + ROPE)
    x, key, table = normal(g, tokens, latent), normal(g, tokens, ROPE), angles(900)
    slots = torch.arange(tokens, device="cuda", dtype=torch.int32)
    caches = [torch.zeros(tokens, 224, dtype=torch.uint8, device="cuda") for _ in range(3)]
    apart, together = query.clone(), query.clone()
    tk.latent4_append(caches[0], x, key, slots, table, slots, interleaved=interleaved,
                      query_rope=query[..., latent:].clone(), query=apart)
    tk.latent4_append(caches[1], x, key, slots, table, slots, interleaved=interleaved,
                      query_rope=together[..., latent:], query=together)
    tk.latent4_append(caches[2], x, key, slots, table, slots, interleaved=interleaved)
    assert torch.equal(apart, together) and all(torch.equal(caches[0], c) for c in caches)


def test_rows_refuses_an_output_that_records_a_gradient():
    cache = Q.random_cache(gen(1), 4, 128)
    at = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    out = torch.zeros(2, 128 + ROPE, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    with pytest.raises(ValueError):
        tk.latent4_rows(cache, at, latent=128, out=out)
    assert not out.any()
    with torch.no_grad():
        tk.latent4_rows(cache, at, latent=128, out=out)
    assert torch.equal(out, tk.latent4_rows(cache, at, latent=128))


@pytest.mark.parametrize("latent", [128, 256, 384, 512])
@pytest.mark.parametrize("count", [0, 1, 9, 1000, 40000])
def test_rows(latent, count):
    g = gen(latent + count)
    cache = Q.random_cache(g, 700, latent, pad=32)
    cache[3, latent // 2 + 2 * ROPE] = 0x7F                 # a scale of NaN, and one with a sign
    cache[4, latent // 2 + 2 * ROPE + 1] = 0xB0
    at = torch.randint(-3, 705, (count,), generator=g, device="cuda").int()
    if count > 8:
        at[:8] = torch.tensor([3, 4, -1, 700, 2 ** 31 - 1, -(2 ** 31), 0, 699], dtype=torch.int32)
    want = torch.zeros(count, latent + ROPE, dtype=torch.float64, device="cuda")
    there = (at >= 0) & (at < 700)
    want[there] = Q.unpack(cache, latent)[at[there].long()]
    got = tk.latent4_rows(cache, at, latent=latent)
    assert got.dtype is torch.bfloat16 and torch.equal(got.double().nan_to_num(7e9), want.nan_to_num(7e9))
    out = torch.full((count, latent + ROPE + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    assert tk.latent4_rows(cache, at, latent=latent, out=out[:, :latent + ROPE]).shape == want.shape
    assert torch.equal(out[:, :latent + ROPE].nan_to_num(7e9), got.nan_to_num(7e9))
    assert (out[:, latent + ROPE:] == 5).all()


# ------------------------------------------------------------------ attention over selected rows

def selected_case(tokens, heads, latent, k, rows, seed, empty=0.1):
    g = gen(seed)
    query, cache = normal(g, tokens, heads, latent + ROPE), Q.random_cache(g, rows, latent)
    sel = torch.randint(0, rows, (tokens, k), generator=g, device="cuda").int()
    sel[torch.rand(tokens, k, generator=g, device="cuda") < empty] = -1
    return query, cache, sel


def check_selected(query, cache, sel, latent, scale=SCALE, **kw):
    out, lse = tk.latent4_attend_selected(query, cache, sel, scale, latent=latent, lse=True, **kw)
    ref, rl, tol, tl = Q.attend(query, Q.unpack(cache, latent), R.visible_selected(sel, cache.shape[0]), scale, latent)
    R.assert_close(out, ref, tol, "out")
    R.assert_close(lse, rl, tl, "lse")
    return out, lse


@pytest.mark.parametrize("k", [0, 1, 2, 127, 128, 129, 255, 256, 400, 1000, 2048])
def test_selected_list_lengths(k):
    check_selected(*selected_case(3, 16, 512, k, 4096, k), 512)


@pytest.mark.parametrize("heads", [1, 3, 8, 16, 17, 20, 32, 33, 40, 64, 65, 96, 128, 200, 256])
@pytest.mark.parametrize("latent", [128, 512])
def test_selected_heads(heads, latent):
    check_selected(*selected_case(5, heads, latent, 300, 1000, heads), latent)


@pytest.mark.parametrize("latent", [128, 256, 384])
@pytest.mark.parametrize("tokens", [1, 40, 200])
@pytest.mark.parametrize("heads", [20, 64])
def test_selected_tokens(tokens, latent, heads):
    check_selected(*selected_case(tokens, heads, latent, 533, 5000, tokens), latent)


def test_selected_many_tokens_of_short_lists():
    check_selected(*selected_case(1500, 16, 128, 70, 3000, 9), 128)


def test_selected_empty_lists_and_empty_places():
    query, cache, sel = selected_case(6, 24, 512, 400, 1000, 1)
    sel[0] = -1                              # nothing at all
    sel[1, :300] = -1                        # whole blocks empty, then rows
    sel[2, 1:] = -1                          # one row
    sel[3, 3], sel[3, 7] = 1000, 2 ** 31 - 1   # past the cache
    sel[4, :] = 17                           # the same row every time
    sel[5, ::2] = -(2 ** 31)
    out, lse = check_selected(query, cache, sel, 512)
    assert torch.count_nonzero(out[0]).item() == 0 and torch.isneginf(lse[0]).all()


@pytest.mark.parametrize("scale", [0.0, 3.0, -0.5, 1e-3, 1e30])
def test_selected_scales(scale):
    # 3.0: scores of hundreds, one row takes nearly all; the maximum rises many times.
    query, cache, sel = selected_case(3, 16, 512, 700, 2000, 4)
    if scale == 1e30:
        query = query * 2.0 ** -100
        query[:, ::2] *= 2.0 ** 10
    check_selected(query, cache, sel, 512, scale=scale)


@pytest.mark.parametrize("heads", [16, 64])
def test_selected_rising_scores(heads):
    # Every list entry's score exceeds the last by about 4: the running maximum moves at every block.
    query, cache, sel = selected_case(2, heads, 512, 700, 700, 5, empty=0.0)
    sel[:] = torch.arange(700, device="cuda").int()
    for r in range(700):
        Q.set_key(cache, r, 512, 0, float(r))
    query[:, :, 512] = 1.0
    query[:, 8:, 512] = -1.0                 # and falls for the other heads
    check_selected(query, cache, sel, 512, scale=4.0)


@pytest.mark.parametrize("power", [-140, -126, -110, -60, -20, 20, 60, 110, 120])
def test_selected_sizes_of_queries(power):
    # A query row's own power of two carries it through FP16; rows of one tile differ in size.
    query, cache, sel = selected_case(2, 24, 256, 300, 900, 6)
    query = (query.double() * 2.0 ** power).to(torch.bfloat16)
    query[:, ::3] = (query[:, ::3].double() * 2.0 ** -9).to(torch.bfloat16)
    query[0, 1] = 0
    # (scores of ordinary size; the scale has to be a float32)
    check_selected(query, cache, sel, 256, scale=min(max(SCALE * 2.0 ** -power, 2.0 ** -126), 2.0 ** 126))


def test_selected_queries_of_values_far_apart():
    # Values down to 2^-40 of the row's largest, against rows where only those count.
    query, cache, sel = selected_case(2, 16, 512, 300, 900, 7)
    query[..., 1:512] = (query[..., 1:512].double() * 2.0 ** -25).to(torch.bfloat16)
    query[..., 0] = 2.0 ** 15
    rows = torch.arange(900, device="cuda")
    Q.set_value(cache, rows, 512, 0, 0, 0x30)
    check_selected(query, cache, sel, 512, scale=2.0 ** 20)


def test_selected_extreme_scales_of_rows():
    # The largest and the smallest scales, with and without sign.
    query, cache, sel = selected_case(3, 16, 256, 300, 900, 8)
    at = 128 + 2 * ROPE
    cache[:300, at:at + 16] = 0x7E
    cache[300:600, at:at + 16] = 0x01
    cache[::7, at + 3] |= 0x80
    check_selected(query, cache, sel, 256, scale=0.01)
    check_selected(query, cache, sel.clamp(min=300, max=599), 256, scale=10.0)


def test_selected_strides_and_given_outputs():
    g = gen(6)
    latent, dim = 256, 320
    query = normal(g, 20, 5, dim + 24)[:, :, 8:8 + dim].transpose(0, 1)
    cache = Q.random_cache(g, 700, latent, pad=96)
    sel = torch.randint(-20, 700, (5, 301), generator=g, device="cuda").int()[:, 3:290]
    out = torch.empty(5, 20, latent, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(5, 20, device="cuda")
    ws = tk.latent4_workspace()
    o, l = tk.latent4_attend_selected(query, cache, sel, SCALE, latent=latent, out=out, lse=lse, workspace=ws)
    assert o is out and l is lse
    ref, rl, tol, tl = Q.attend(query, Q.unpack(cache, latent), R.visible_selected(sel, 700), SCALE, latent)
    R.assert_close(out, ref, tol, "out")
    R.assert_close(lse, rl, tl, "lse")
    o, l = tk.latent4_attend_selected(query, cache, sel, SCALE, latent=latent)
    assert torch.equal(o, out) and l is None
    one = tk.latent4_attend_selected(query[:1], cache, sel[:1], SCALE, latent=latent)[0]
    R.assert_close(one, ref[:1], tol[:1], "one token")
    check_selected(query[:, :1].expand(5, 20, dim), cache, sel, latent)       # broadcast over its heads


def test_selected_no_tokens_and_no_cache():
    query, cache, sel = selected_case(2, 16, 512, 100, 300, 7)
    out, lse = tk.latent4_attend_selected(query[:0], cache, sel[:0], SCALE, lse=True)
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16)
    out, lse = tk.latent4_attend_selected(query, cache[:0], sel, SCALE, lse=True)
    assert torch.count_nonzero(out).item() == 0 and torch.isneginf(lse).all()


def test_rows_past_32_bit_offsets():
    # 5 GB of cache: byte offsets of the last rows pass 2^32.
    rows, latent = 12_500_000, 512
    cache = torch.empty(rows, 416, dtype=torch.uint8, device="cuda")
    g = gen(8)
    cache[-320:], cache[:320] = Q.random_cache(g, 320, latent), Q.random_cache(g, 320, latent)
    sel = torch.randint(0, 300, (2, 256), generator=g, device="cuda").int()
    sel[:, ::2] = rows - 1 - sel[:, ::2]
    query = normal(g, 2, 16, 576)
    small = torch.cat((cache[:320], cache[-320:]))
    there = torch.where(sel < 320, sel, sel - rows + 640)
    out, lse = tk.latent4_attend_selected(query, cache, sel, SCALE, lse=True)
    ref, rl, tol, tl = Q.attend(query, Q.unpack(small, latent), R.visible_selected(there, 640), SCALE, latent)
    R.assert_close(out, ref, tol, "out")
    R.assert_close(lse, rl, tl, "lse")
    pages = rows // 64
    table = torch.tensor([[pages - 1, 3, pages - 5, 0], [1, pages - 2, 4, pages - 3]], dtype=torch.int32, device="cuda")
    valid = torch.tensor([250, 251, 200, 201], dtype=torch.int32, device="cuda")
    query = normal(g, 4, 16, 576)
    out, lse = tk.latent4_attend_paged(query, cache, valid, table, SCALE, lse=True, rows_per_request=2)
    moved = torch.where(table < 5, table, table - pages + 10)
    ref, rl, tol, tl = Q.attend(query, Q.unpack(small, latent), R.visible_paged(valid, moved, 256, 64, 64, 2, 640),
                                SCALE, latent)
    # (12,500,000 is not a whole number of pages: the last page ends before the cache does.)
    assert rows % 64 == 32 or rows % 64 == 0
    if rows % 64 == 0:
        R.assert_close(out, ref, tol, "out")
        R.assert_close(lse, rl, tl, "lse")
    back = tk.latent4_rows(cache, sel[0])
    assert torch.equal(back.double(), Q.unpack(small, latent)[there[0].long()])
    slot = torch.tensor([rows - 1, 0], dtype=torch.int32, device="cuda")
    x = normal(g, 2, latent)
    tk.latent4_append(cache, x, normal(g, 2, ROPE), torch.zeros_like(slot), angles(2), slot)
    code, scale = Q.quantise(x.double())
    got = torch.stack((cache[-1], cache[0]))
    assert torch.equal(got[:, 384:].long(), scale)


# ------------------------------------------------------------------ attention over pages

def paged_case(lens, q, heads, latent, page, seed, block_rows=None, width=None):
    """lens: context length of each request, its q new tokens the last of them."""
    g = gen(seed)
    block_rows = block_rows or page
    n = len(lens)
    pages = -(-max(max(lens), width or 1) // page)
    table = torch.randperm(n * pages + 3, generator=g, device="cuda")[:n * pages].view(n, pages).int()
    cache = Q.random_cache(g, (n * pages + 3) * block_rows, latent)
    valid = torch.tensor([max(0, ln - q + 1 + j) for ln in lens for j in range(q)], dtype=torch.int32, device="cuda")
    return normal(g, n * q, heads, latent + ROPE), cache, valid, table, dict(page_size=page, block_rows=block_rows,
                                                                             rows_per_request=q)


def check_paged(query, cache, valid, table, kw, latent, scale=SCALE):
    out, lse = tk.latent4_attend_paged(query, cache, valid, table, scale, latent=latent, lse=True, **kw)
    width = kw.get("width") or table.shape[1] * kw["page_size"]
    visible = R.visible_paged(valid, table, width, kw["page_size"], kw["block_rows"], kw["rows_per_request"],
                              cache.shape[0])
    ref, rl, tol, tl = Q.attend(query, Q.unpack(cache, latent), visible, scale, latent)
    R.assert_close(out, ref, tol, "out")
    R.assert_close(lse, rl, tl, "lse")
    return out, lse


@pytest.mark.parametrize("length", [1, 2, 63, 127, 128, 129, 256, 257, 1000, 9000])
def test_paged_lengths(length):
    check_paged(*paged_case([length], 1, 16, 512, 64, length), 512)


@pytest.mark.parametrize("q,heads", [(1, 1), (2, 1), (3, 16), (4, 20), (5, 33), (7, 128), (70, 1), (33, 3), (2, 96),
                                     (129, 8), (200, 2)])
@pytest.mark.parametrize("latent", [128, 512])
def test_paged_chunks(q, heads, latent):
    check_paged(*paged_case([q + 170, max(1, q // 2), 333], q, heads, latent, 64, q * heads), latent)


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


@pytest.mark.parametrize("rows", [150, 190, 63, 65])
def test_paged_last_page_ends_with_the_cache(rows):
    query, cache, valid, table, kw = paged_case([256, 100], 2, 16, 256, 64, 83)
    table[0], table[1] = torch.tensor([2, 0, 1, 3]), torch.tensor([1, 2, 0, 3])
    check_paged(query, cache[:rows], valid, table, kw, 256)


def test_paged_one_long_context():
    check_paged(*paged_case([50_001], 2, 16, 512, 64, 17), 512)
    check_paged(*paged_case([30_001], 1, 128, 512, 64, 18), 512)


def test_paged_rows_per_request_past_the_tokens():
    query, cache, valid, table, kw = paged_case([90], 3, 16, 128, 64, 19)
    want, _ = check_paged(query, cache, valid, table, kw, 128)
    got, _ = tk.latent4_attend_paged(query, cache, valid, table, SCALE, latent=128,
                                     **dict(kw, rows_per_request=2 ** 31 - 1))
    assert torch.equal(got, want)


# ------------------------------------------------------------------ what is not finite

@pytest.mark.parametrize("heads", [1, 16, 64])
def test_paged_what_a_token_may_not_see_does_not_reach_it(heads):
    # Stale rows past the context and a later token of the chunk, of scales that are NaN or key parts that are not finite.
    q, latent = 6, 512
    for bad in ("scale", float("nan"), float("inf"), float("-inf")):
        query, cache, valid, table, kw = paged_case([200, 167], q, heads, latent, 64, 16)
        query[:, :, latent] = query[:, :, latent].abs() + 0.5
        gone = []
        for r, n in enumerate((200, 167)):
            i = torch.arange(n, table.shape[1] * 64, device="cuda")
            last = torch.tensor([int(table[r, (n - 2) // 64]) * 64 + (n - 2) % 64], device="cuda")
            gone.append(torch.cat((table[r].long()[i // 64] * 64 + i % 64, last)))   # past the context; token q - 2
        gone = torch.cat(gone)
        visible = R.visible_paged(valid, table, table.shape[1] * 64, 64, 64, q, cache.shape[0])
        ref, rl, tol, tl = Q.attend(query, Q.unpack(cache, latent), visible, SCALE, latent)
        if bad == "scale":
            cache[gone, latent // 2 + 2 * ROPE:] = 0x7F
        else:
            Q.set_key(cache, gone, latent, 0, bad)
            cache[gone, latent // 2 + 2 * ROPE + 3] = 0x7F
        out, lse = tk.latent4_attend_paged(query, cache, valid, table, SCALE, latent=latent, lse=True, **kw)
        for r in range(2):
            s = slice(r * q, r * q + q - 2)
            R.assert_close(out[s], ref[s], tol[s], "out")
            R.assert_close(lse[s], rl[s], tl[s], "lse")
            assert torch.isnan(out[r * q + q - 2:(r + 1) * q]).all()


def test_selected_rows_that_nobody_sees_may_hold_anything():
    query, cache, sel = selected_case(4, 16, 512, 130, 600, 2)
    seen = torch.zeros(600, dtype=torch.bool, device="cuda")
    seen[sel[sel >= 0].long()] = True
    clean = check_selected(query, cache, sel, 512)
    cache[~seen] = 0x7F
    cache[0 if not seen[0] else int(torch.nonzero(~seen)[0])] = 0xFF
    got = tk.latent4_attend_selected(query, cache, sel, SCALE, lse=True)
    assert all(torch.equal(a, b) for a, b in zip(clean, got))


@pytest.mark.parametrize("heads", [4, 16, 64])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_paged_a_bad_query_row_stays_alone(heads, bad):
    query, cache, valid, table, kw = paged_case([230, 171], 5, heads, 256, 64, 18)
    clean, cl = check_paged(query, cache, valid, table, kw, 256)
    query[1, 2] = bad
    query[8, 0, 300] = bad
    out, lse = tk.latent4_attend_paged(query, cache, valid, table, SCALE, latent=256, lse=True, **kw)
    touched = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    touched[1, 2] = touched[8, 0] = True
    assert torch.equal(out[~touched], clean[~touched]) and torch.equal(lse[~touched], cl[~touched])
    assert not torch.isfinite(out[1, 2]).any()


@pytest.mark.parametrize("form,tokens,length", [("listed", 1, 2048), ("listed", 1, 30000), ("listed", 200, 700),
                                                ("paged", 1, 2048), ("paged", 1, 30000), ("paged", 3, 700)])
@pytest.mark.parametrize("first,blocks", [(0, 1), (0, 2), (0, 5), (3, 7), (0, 10 ** 6)])
def test_scores_of_minus_infinity_weigh_nothing(form, tokens, length, first, blocks):
    heads, latent = 16, 256
    query, cache, _ = selected_case(tokens, heads, latent, 1, -(-length // 64) * 64, 50)
    if form == "listed":
        order = torch.randperm(length, generator=gen(50), device="cuda").int()
        lists = order.expand(tokens, length).contiguous()
    else:
        table = torch.randperm(cache.shape[0] // 64, generator=gen(50), device="cuda").int()
        at = torch.arange(length, device="cuda")
        order = table[at // 64] * 64 + (at % 64).int()
        valid = torch.full((tokens,), length, dtype=torch.int32, device="cuda")
    order = order.long()
    gone = torch.zeros(length, dtype=torch.bool, device="cuda")
    gone[first * 128:(first + blocks) * 128] = True
    query[..., latent] = 1.0
    Q.set_key(cache, torch.arange(cache.shape[0], device="cuda"), latent, 0, 0.0)
    Q.set_key(cache, order[gone], latent, 0, float("-inf"))
    if form == "listed":
        out, lse = tk.latent4_attend_selected(query, cache, lists, SCALE, latent=latent, lse=True)
    else:
        out, lse = tk.latent4_attend_paged(query, cache, valid, table[None], SCALE, latent=latent, lse=True,
                                           rows_per_request=tokens)
    if gone.all():
        assert torch.count_nonzero(out).item() == 0 and torch.isneginf(lse).all()
        return
    query[..., latent] = 0.0
    Q.set_key(cache, order[gone], latent, 0, 0.0)
    ref, rl, tol, tl = Q.attend(query, Q.unpack(cache, latent), [order[~gone]] * tokens, SCALE, latent)
    R.assert_close(out, ref, tol, "out")
    R.assert_close(lse, rl, tl, "lse")


def test_a_score_of_minus_infinity_masks_whatever_its_row_holds():
    # A row at -inf for half of the heads by its key part, whose last values are NaN only in the others' eyes: a scale of
    # NaN makes every score of it NaN, so it reaches all that see it and none else.
    query, cache, sel = selected_case(3, 16, 256, 300, 500, 3, empty=0.0)
    sel[sel == 123] = 124
    sel[1, 50] = 123
    Q.set_key(cache, 123, 256, 0, float("inf"))
    query[:, :8, 256], query[:, 8:, 256] = -1.0, 1.0
    out, lse = tk.latent4_attend_selected(query, cache, sel, SCALE, latent=256, lse=True)
    rest = sel.clone()
    rest[1, 50] = -1
    ref, rl, tol, tl = Q.attend(query, Q.unpack(cache, 256), R.visible_selected(rest, 500), SCALE, 256)
    R.assert_close(out[:, :8], ref[:, :8], tol[:, :8], "out")
    R.assert_close(lse[:, :8], rl[:, :8], tl[:, :8], "lse")
    assert torch.isnan(out[1, 8:]).all() and torch.isfinite(out[0]).all() and torch.isfinite(out[2]).all()
    cache[123, 128 + 2 * ROPE + 2] = 0x7F
    out, _ = tk.latent4_attend_selected(query, cache, sel, SCALE, latent=256)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[0]).all() and torch.isfinite(out[2]).all()


# ------------------------------------------------------------------ the dealing of work

@pytest.mark.parametrize("k", [128, 250, 700, 1024, 1100])
@pytest.mark.parametrize("tokens,heads", [(1, 16), (2, 128), (9, 33)])
def test_selected_short_work_in_clusters(tokens, heads, k):
    check_selected(*selected_case(tokens, heads, 384, k, 3000, k + tokens), 384)


@pytest.mark.parametrize("lens", [[1500] * 140, [1500 - 9 * i for i in range(60)] + [1500] * 80, [1500] * 100 + [1] * 40,
                                  [2000 + i for i in range(152)]])
@pytest.mark.parametrize("heads", [16, 64])
def test_pages_of_about_as_many_tiles_as_sms(lens, heads):
    query, cache, valid, table, kw = paged_case(lens, 1, heads, 128, 64, 76)
    valid[7] = 0
    check_paged(query, cache, valid, table, kw, 128)


def test_a_long_tile_among_many_short_ones():
    check_paged(*paged_case([40000] + [500] * 99, 1, 16, 256, 64, 71), 256)
    check_paged(*paged_case([300] * 60 + [30001] + [77] * 30, 1, 64, 128, 64, 72), 128)


def test_many_tiles_of_64_rows_of_the_widest_latent():
    # More tiles than SMs: several pieces a CTA, tiles split between CTAs, a last tile of few rows.
    check_selected(*selected_case(230, 70, 512, 333, 3000, 73), 512)
    lens = [200 + (i * 37) % 190 for i in range(90)]
    query, cache, valid, table, kw = paged_case(lens, 3, 67, 512, 64, 74)
    check_paged(query[:268], cache, valid[:268], table, kw, 512)


def test_ways_of_dealing_agree():
    query, cache, sel = selected_case(1, 16, 256, 900, 4000, 40, empty=0.0)
    check_selected(query, cache, sel, 256)
    many, lm = tk.latent4_attend_selected(query.expand(400, 16, 320), cache, sel.expand(400, 900).contiguous(), SCALE,
                                          latent=256, lse=True)
    paged, lp = tk.latent4_attend_paged(query, cache, torch.tensor([900], dtype=torch.int32, device="cuda"), sel, SCALE,
                                        page_size=1, latent=256, lse=True)
    ref, rl, tol, tl = Q.attend(query, Q.unpack(cache, 256), R.visible_selected(sel, 4000), SCALE, 256)
    for got, lse in ((many, lm), (paged, lp)):
        R.assert_close(got, ref.expand(got.shape), tol.expand(got.shape), "out")
        R.assert_close(lse, rl.expand(lse.shape), tl.expand(lse.shape), "lse")


# ------------------------------------------------------------------ streams, repeats, the step together

def test_repeats_are_bit_equal_and_streams_are_kept():
    query, cache, sel = selected_case(9, 128, 512, 2048, 30000, 20)
    first = tk.latent4_attend_selected(query, cache, sel, SCALE, lse=True)
    for _ in range(5):
        again = tk.latent4_attend_selected(query, cache, sel, SCALE, lse=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [tk.latent4_attend_selected(query, cache, sel, SCALE, lse=True, stream=s) for s in (side, None, side, None)]
    torch.cuda.synchronize()
    for again in got:
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_two_calls_at_once():
    # Split tiles and clusters of both forms on two streams, eagerly and as graphs replayed side by side, each call
    # with scratch of its own; a shared one serves calls that follow each other on one stream.
    query, cache, sel = selected_case(9, 64, 512, 2048, 9000, 31)
    table = torch.arange(140, device="cuda", dtype=torch.int32)[None]
    lens = torch.full((9,), 8960, dtype=torch.int32, device="cuda") - torch.arange(9, device="cuda").flip(0).int()
    shared = tk.latent4_workspace()

    def one(workspace=None):
        return tk.latent4_attend_selected(query, cache, sel, SCALE, lse=True, workspace=workspace)

    def other(workspace=None):
        return tk.latent4_attend_paged(query, cache, lens, table, SCALE, rows_per_request=9, lse=True,
                                       workspace=workspace)

    want = (*one(), *other())
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graphs, held = [], []
    for call in (one, other):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append([call() for _ in range(3)])
        graphs.append(graph)
    torch.cuda.synchronize()
    eager = [[], []]
    for i in range(12):
        for k, call in enumerate((one, other)):
            with torch.cuda.stream(streams[k]):
                eager[k].append(call())
                graphs[k].replay()
    torch.cuda.synchronize()
    both = [(one(shared), other(shared)) for _ in range(5)]
    torch.cuda.synchronize()
    for k in range(2):
        for got in (*eager[k], *held[k], *(b[k] for b in both)):
            assert torch.equal(got[0], want[2 * k]) and torch.equal(got[1], want[2 * k + 1])


@pytest.mark.parametrize("latent", [128, 512])
def test_a_paged_step_over_pages_in_four_bits(latent):
    """The operators as a server uses them, captured once and replayed: tables and slots, append, selection from the
    indexer's scores, attention over the selection and over everything. Requests begin, idle, grow and end."""
    g = gen(22)
    heads, n, q, pages, page = 16, 5, 2, 8, 64
    cache = torch.zeros((n * pages + 2) * page, tk.latent4_row_bytes(latent), dtype=torch.uint8, device="cuda")
    mirror = cache.clone()
    table = torch.full((n, pages), -1, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(n, dtype=torch.int32, device="cuda")
    new = torch.zeros_like(lengths)
    free = torch.randperm(n * pages + 2, generator=g, device="cuda").int()
    count = torch.tensor([n * pages + 2], dtype=torch.int32, device="cuda")
    x, key = normal(g, n * q, latent), normal(g, n * q, ROPE)
    query, query_rope = normal(g, n * q, heads, latent + ROPE), normal(g, n * q, heads, ROPE)
    scores, turn = normal(g, n * q, pages * page), angles(pages * page)
    weight = 1 + normal(g, latent) / 8

    def step():
        at = tk.page_step(table, lengths, new, free, count, rows_per_request=q)
        tk.latent4_append(cache, x, key, at.positions, turn, at.slots, weight=weight, query_rope=query_rope, query=query)
        rows = tk.select(scores, at.valid_len, 128, tk.TOKEN, table, page, rows_per_request=q)
        some = tk.latent4_attend_selected(query, cache, rows, SCALE, latent=latent, lse=True)
        whole = tk.latent4_attend_paged(query, cache, at.valid_len, table, SCALE, latent=latent, lse=True,
                                        rows_per_request=q)
        return at, rows, some, whole

    step()                                   # (nothing new: warms up what a capture may not)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        at, rows, some, whole = step()
    held = [0] * n
    for i in range(300):
        ask = [2 if (i + r) % 3 else 1 for r in range(n)]
        if i % 40 == 39:
            ask[i // 40 % n] = -1
        if i % 7 == 3:
            ask[(i // 7) % n] = 0
        new.copy_(torch.tensor(ask, dtype=torch.int32))
        x.copy_(normal(g, n * q, latent))
        key.copy_(normal(g, n * q, ROPE))
        scores.copy_(normal(g, n * q, pages * page))
        graph.replay()
        for r in range(n):
            # (a request that is full stays as it is)
            held[r] = 0 if ask[r] < 0 else held[r] + (ask[r] if held[r] + ask[r] <= pages * page else 0)
        # The appended rows, by one eager call into a second cache.
        tk.latent4_append(mirror, x, key, at.positions, turn, at.slots, weight=weight)
        if i % 50 != 17:
            continue
        assert lengths.tolist() == held and torch.equal(cache, mirror)
        values = Q.unpack(cache, latent)
        for got, visible in ((some, R.visible_selected(rows, cache.shape[0])),
                             (whole, R.visible_paged(at.valid_len, table, pages * page, page, page, q, cache.shape[0]))):
            assert [v.numel() for v in visible] == [min(v, 128 if got is some else 9999) for v in at.valid_len.tolist()]
            ref, rl, tol, tl = Q.attend(query, values, visible, SCALE, latent)
            R.assert_close(got[0], ref, tol, "out")
            R.assert_close(got[1], rl, tl, "lse")


# ------------------------------------------------------------------ refusals

def test_refusals():
    query, cache, sel = selected_case(2, 16, 512, 100, 300, 30)
    valid = torch.ones(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")

    def selected(q=query, c=cache, s=sel, **kw):
        return tk.latent4_attend_selected(q, c, s, SCALE, **kw)

    def paged(q=query, c=cache, v=valid, t=table, **kw):
        return tk.latent4_attend_paged(q, c, v, t, SCALE, **kw)

    wide = torch.zeros(300, 576, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: selected(query.float()), lambda: selected(query.cpu()), lambda: selected(s=sel.long()),
                 lambda: paged(v=valid.long()), lambda: paged(c=cache.char()), lambda: paged(c=wide),
                 lambda: selected(c=wide), lambda: tk.latent_attend_selected(query, cache, sel, SCALE),
                 lambda: tk.latent4_rows(wide, valid), lambda: tk.latent4_rows(cache, valid.long()),
                 lambda: tk.latent4_rows(cache, 3)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: selected(latent=256), lambda: selected(latent=500), lambda: selected(query[..., :512]),
                 lambda: selected(s=sel[:1]), lambda: selected(c=cache[:, :384]),
                 lambda: selected(out=torch.empty(2, 16, 512, device="cuda")),
                 lambda: selected(workspace=torch.empty(64, device="cuda")), lambda: paged(v=valid[:1]),
                 lambda: paged(page_size=48), lambda: paged(width=257), lambda: paged(rows_per_request=0),
                 lambda: tk.latent4_rows(cache, valid, latent=256), lambda: tk.latent4_rows(cache, sel),
                 lambda: tk.latent4_rows(cache, valid, out=torch.empty(2, 576, device="cuda")),
                 lambda: tk.latent4_rows(cache, valid, out=torch.empty(3, 576, dtype=torch.bfloat16, device="cuda")),
                 lambda: tk.latent4_row_bytes(100)):
        with pytest.raises(ValueError):
            call()
    pages = torch.zeros(2, 9000, dtype=torch.int32, device="cuda")     # long enough to need scratch
    off = torch.zeros(400 * 448, dtype=torch.uint8, device="cuda")
    bent = torch.zeros(9, 584, dtype=torch.bfloat16, device="cuda")
    for call, status in ((lambda: paged(t=pages, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), 1),
                         (lambda: paged(block_rows=32), 1),
                         (lambda: tk.latent4_attend_selected(query, cache, sel, float("nan")), 1),
                         (lambda: selected(c=off[16:16 + 299 * 416].view(299, 416)), 2),
                         (lambda: selected(c=off.view(400, 448)[:, :416].as_strided((300, 416), (432, 1))), 2),
                         (lambda: tk.latent4_rows(off[16:16 + 299 * 416].view(299, 416), valid), 2),
                         (lambda: tk.latent4_rows(cache, valid, out=bent.flatten()[4:4 + 1160].view(2, 580)[:, :576]), 2)):
        with pytest.raises(tk.TopkError) as e:
            call()
        assert e.value.status == status
    x, key, pos = normal(gen(1), 2, 512), normal(gen(2), 2, ROPE), valid
    for kw in (dict(latent=x[:, :500]), dict(latent=x[:, :256]), dict(key_rope=key[:, :32]),
               dict(cos_sin=angles(4)[:, :32]), dict(slots=pos[:1]), dict(query=query), dict(weight=x[0, :256])):
        args = dict(cache=cache, latent=x, key_rope=key, positions=pos, cos_sin=angles(4), slots=pos)
        with pytest.raises(ValueError):
            tk.latent4_append(**{**args, **kw})
    with pytest.raises(TypeError):
        tk.latent4_append(wide, x, key, pos, angles(4), pos)
    with pytest.raises(ValueError, match="gradient"):
        selected(query.clone().requires_grad_())
    with pytest.raises(ValueError, match="gradient"):
        tk.latent4_append(cache, x.clone().requires_grad_(), key, pos, angles(4), pos)


# ------------------------------------------------------------------ the size of the errors

@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("length", [100, 2048])
def test_errors_are_of_one_rounding(heads, length):
    # Weights in FP16 leave 2^-11 / sqrt 3 of the output's mean square, the output's own rounding to BF16 2^-8 / sqrt 3:
    # together 2^-8 sqrt((1 + 2^-6) / 3), with a tenth for the sample.
    query, cache, sel = selected_case(40, heads, 512, length, 9000, 90)
    values = Q.unpack(cache, 512)
    out, _ = tk.latent4_attend_selected(query, cache, sel, SCALE)
    ref = Q.attend(query, values, R.visible_selected(sel, 9000), SCALE, 512)[0]
    most = 1.1 * ((1 + 2.0 ** -6) / 3) ** 0.5 * 2.0 ** -8
    assert ((out.double() - ref).pow(2).mean() / ref.pow(2).mean()).sqrt().item() < most
