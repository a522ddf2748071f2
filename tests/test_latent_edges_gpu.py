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
