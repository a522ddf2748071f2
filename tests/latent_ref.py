"""The latent-cache operators in 64 bits, written from their formulas, and the
error bounds the kernels are held to."""
from __future__ import annotations

import torch

ROPE = 64
U16 = 2.0 ** -8      # half a unit in the last place of BF16 (8 significant bits), relative
INF = float("inf")


def rotate(x, angles, interleaved=True):
    """x [..., 64] (float64) by angles [..., 64] (32 cosines, 32 sines)."""
    cos, sin = angles[..., :32], angles[..., 32:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def norm(x, weight, eps):
    x = x.double()
    return x * weight.double() / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()


def visible_selected(selected, cache_rows):
    """Per token: the listed rows that lie inside the cache."""
    return [row[(row >= 0) & (row < cache_rows)].long() for row in selected]


def visible_paged(valid_len, table, width, page, block_rows, q, cache_rows):
    out = []
    for t, n in enumerate(valid_len.tolist()):
        i = torch.arange(max(0, min(n, width)), device=table.device)
        row = table[t // q].long()[i // page] * block_rows + i % page
        out.append(row[(row >= 0) & (row < cache_rows)])
    return out


def attend(query, cache, visible, scale, latent):
    """(out, lse, tolerance of out, tolerance of lse), each row from its visible
    cache rows alone.

    The kernels round each p_j (relative U16) and the result (U16) to BF16 and
    hold scores, sums and products in 32 bits. Let D be the largest error of a
    score: 36 steps of 16 products with at most 2^-23 of the partial sum each
    come to less than 2^-17 of sum |q k|; twice that covers the scale's
    rounding and the exponent's. A score error changes p_j by 2 D relative at
    most (numerator and sum), so |out - ref| <= U16 |ref| + (U16 + 2 D)
    sum p |c|, with 10 % for products of these and 2^-100 for what underflows.
    The sums of p in 32 bits: 2^-20 relative covers the exponentials' 2^-22 and
    the additions of at most 2^12 terms per partial sum in four lanes.
    """
    tokens, heads, _ = query.shape
    dev = query.device
    out = torch.zeros(tokens, heads, latent, dtype=torch.float64, device=dev)
    lse = torch.full((tokens, heads), -INF, dtype=torch.float64, device=dev)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for t, rows in enumerate(visible):
        if rows.numel() == 0:
            continue
        q, keys = query[t].double(), cache[rows].double()
        s = q @ keys.T * scale
        m = s.amax(1, keepdim=True)
        p = torch.exp(s - m)
        total = p.sum(1, keepdim=True)
        p = p / total
        lse[t] = (m + total.log())[:, 0]
        out[t] = p @ keys[:, :latent]
        d = (q.abs() @ keys.abs().T).amax(1, keepdim=True) * abs(scale) * 2.0 ** -16
        tol[t] = 1.1 * (U16 * out[t].abs() + (U16 + 2 * d + 2.0 ** -20) * (p @ keys[:, :latent].abs())) + 2.0 ** -100
        tol_lse[t] = d[:, 0] + 2.0 ** -20 * (1 + lse[t].abs())
    return out, lse, tol, tol_lse


def assert_close(got, ref, tol, what=""):
    """got within tol of ref where ref is finite; equal infinities; NaN where NaN."""
    got = got.double()
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    rest = ~fine & ~torch.isnan(ref)
    assert torch.equal(got[rest], ref[rest]), f"{what}: infinities differ"
    over = (got - ref).abs()[fine] - tol[fine]
    assert over.numel() == 0 or over.max().item() <= 0, (
        f"{what}: off by {(got - ref).abs()[fine].max().item():.3g}, {(over > 0).sum().item()} of "
        f"{over.numel()} values over their bound by up to {over.max().item():.3g}")
