"""The 4-bit latent cache's operators at the ends of their ranges, against their formulas in 64 bits."""
from __future__ import annotations

import pytest
import torch

import exact_bf16_top_gb300 as tk
import latent4_ref as Q
import latent_ref as R
from test_latent_gpu import ROPE, clean_status, gen  # noqa: F401

pytestmark = pytest.mark.gpu

LN2 = 0.6931471824645996     # the float32 next to ln 2: times it, a score is its own value in log2 units


# ------------------------------------------------------------------ large scores

def check_large(query, cache, scale, latent, selected=None, valid=None, table=None, q=1):
    """Attention whose scores are float32 numbers, exact in the kernel, and either equal or at least 4 apart.

    A weight p is then off by the exponential's 2^-22 and, of scores a few tens apart, by the difference of
    float32's ln 2 (2^-24 of it): 2^-16 covers both. Its rounding to FP16: 2^-11 of itself, or 2^-33 of the row's
    sum (latent4_ref.attend). The result is rounded to BF16 once; 10 % for products of these.
    """
    if selected is not None:
        out, lse = tk.latent4_attend_selected(query, cache, selected, scale, latent=latent, lse=True)
        visible = R.visible_selected(selected, cache.shape[0])
    else:
        out, lse = tk.latent4_attend_paged(query, cache, valid, table, scale, rows_per_request=q, latent=latent, lse=True)
        visible = R.visible_paged(valid, table, table.shape[1] * 64, 64, 64, q, cache.shape[0])
    values = Q.unpack(cache, latent)
    ref, rl, _, _ = Q.attend(query, values, visible, scale, latent)
    tol = torch.zeros_like(ref)
    for t, rows in enumerate(visible):
        c = values[rows, :latent].abs()
        p = torch.softmax(query[t].double() @ values[rows].T * scale, 1)
        tol[t] = 1.1 * (R.U16 * ref[t].abs() + (2.0 ** -11 + 2.0 ** -16) * (p @ c) + 2.0 ** -33 * c.sum(0))
    R.assert_close(out, ref, tol, "out")
    R.assert_close(lse, rl, 2.0 ** -20 * (1 + rl.abs()), "lse")


def large_case(g, heads, latent, rows):
    """A cache without key parts, and queries of 1 and -1 on the first value of theirs."""
    cache = Q.random_cache(g, rows, latent)
    cache[:, latent // 2:latent // 2 + 2 * ROPE] = 0
    query = torch.zeros(4, heads, latent + ROPE, dtype=torch.bfloat16, device="cuda")
    query[:, :, latent] = 1.0
    query[:, 1::2, latent] = -1.0
    return cache, query


def set_keys(cache, latent, column, values):
    at = latent // 2 + 2 * column
    cache[:, at:at + 2] = values.to(torch.bfloat16).view(torch.uint8).view(-1, 2)


def check_forms(query, cache, latent, order):
    """Both forms over the rows of `order`, 700 of them."""
    check_large(query, cache, LN2, latent, selected=order.int().repeat(4, 1))
    table = torch.arange(22, dtype=torch.int32, device="cuda").view(2, 11)
    paged = torch.empty_like(cache)
    paged[:704], paged[704:] = cache[order], cache[order]
    valid = torch.tensor([700, 701, 332, 333], dtype=torch.int32, device="cuda")
    check_large(query, paged, LN2, latent, valid=valid, table=table, q=2)


@pytest.mark.parametrize("heads", [3, 16, 32, 64])
@pytest.mark.parametrize("power", range(16, 31))
def test_large_scores(heads, power):
    # Scores of 2^power to 2^(power + 1) in log2 units, of both signs: float32 numbers that lie up to 128 apart.
    # They are rounded to 8 bits here, so they are equal or so far apart that the smaller weighs nothing.
    g, latent = gen(power), 256
    cache, query = large_case(g, heads, latent, 1408)
    set_keys(cache, latent, 0, torch.randint(128, 256, (1408,), generator=g, device="cuda") * 2.0 ** (power - 7))
    rows = torch.randperm(1408, generator=g, device="cuda")[:704]
    check_forms(query, cache, latent, rows)
    key = cache[rows, latent // 2:latent // 2 + 2].contiguous().view(torch.bfloat16)[:, 0]
    check_forms(query, cache, latent, rows[key.float().argsort()])        # the maximum rises at every block
    check_forms(query, cache, latent, rows[key.float().argsort(descending=True)])


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("rise", [4, 8, 12, 15, 16, 17, 24])
@pytest.mark.parametrize("power", range(18, 28))
def test_large_scores_that_rise(heads, rise, power):
    # One row of every 128 has a score of 2^power and as many rises as blocks precede it; the others weigh nothing.
    if rise % 2.0 ** (power - 23):
        pytest.skip("not a float32 number beside 2^power")
    g, latent = gen(power), 256
    cache, query = large_case(g, heads, latent, 1408)
    query[:, :, latent], query[:, :, latent + 1] = 1.0, 1.0
    at = torch.arange(1408, device="cuda")
    block = at % 704 // 128
    most = at % 704 % 128 == (block * 37 + 5) % 60
    set_keys(cache, latent, 0, torch.full((1408,), 2.0 ** power, device="cuda"))
    set_keys(cache, latent, 1, torch.where(most, block * float(rise), -4096.0))
    check_forms(query, cache, latent, at[:704])


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("power", [21, 24, 26, 27, 28])
def test_large_scores_whose_last_bit_is_odd(heads, power):
    # One score for all rows of a list, in one block and in many: less 8 it may round to 16 below itself.
    g, latent = gen(power), 256
    cache, query = large_case(g, heads, latent, 1408)
    query[:, :, latent], query[:, :, latent + 1] = 1.0, 1.0
    set_keys(cache, latent, 0, torch.full((1408,), 2.0 ** power, device="cuda"))
    order = torch.arange(704, device="cuda")
    for odd in (1, 3, 7, 101):
        set_keys(cache, latent, 1, torch.full((1408,), odd * 2.0 ** (power - 23), device="cuda"))
        check_forms(query, cache, latent, order)
        check_large(query, cache, LN2, latent, selected=order[:100].int().repeat(4, 1))
        query.neg_()
