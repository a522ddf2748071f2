"""The 4-bit latent cache's format and operators in 64 bits, written from their
formulas, and the error bounds the kernels are held to."""
from __future__ import annotations

import torch

import latent_ref as R

ROPE = 64
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def e4m3(code):
    """Value (float64) of e4m3 codes: 4 bits of exponent (bias 7), 3 of fraction, 0x7F NaN."""
    code = code.long()
    e, f = (code >> 3) & 15, code & 7
    v = torch.where(e > 0, (8 + f).double() * torch.exp2((e - 10).double()), f.double() * 2.0 ** -9)
    v = torch.where((code & 0x7F) == 0x7F, float("nan"), v)
    return torch.where(code > 127, -v, v)


def unpack(cache, latent):
    """float64 [rows, latent + 64] of a cache's bytes."""
    level = torch.tensor(LEVELS, dtype=torch.float64, device=cache.device)
    codes = cache[:, :latent // 2].long()
    codes = torch.stack((codes & 15, codes >> 4), 2).flatten(1)
    v = torch.where(codes > 7, -level[codes & 7], level[codes & 7])
    key = cache[:, latent // 2:latent // 2 + 2 * ROPE].contiguous().view(torch.bfloat16).double()
    at = latent // 2 + 2 * ROPE
    return torch.cat((v * e4m3(cache[:, at:at + latent // 16]).repeat_interleave(16, 1), key), 1)


def nearest(x, grid):
    """Index of the nearest of an ascending grid's values, of two at the same distance the even one."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, grid.numel() - 1)
    lo = hi - 1
    d = (grid[hi] - x) - (x - grid[lo])
    return torch.where((d < 0) | ((d == 0) & (hi % 2 == 0)), hi, lo)


def quantise(v):
    """(codes without sign, scale codes) of float64 values [n, latent]; blocks that are not finite get scale 0x7F."""
    n, latent = v.shape
    b = v.abs().view(n, latent // 16, 16)
    odd = ~torch.isfinite(b).all(2)
    b = torch.where(odd[..., None], 0.0, b)
    grid = e4m3(torch.arange(0x7F, device=v.device))
    scale = nearest((b.amax(2) / 6).clamp(max=448.0), grid).clamp(min=1)
    level = torch.tensor(LEVELS, dtype=torch.float64, device=v.device)
    code = nearest((b / grid[scale][..., None]).clamp(max=6.0), level)
    return code.view(n, latent), torch.where(odd, 0x7F, scale)


def random_cache(g, rows, latent, pad=0):
    """Any codes, scales between 2^-4 and 2^-1, normal key parts; `pad` more bytes a row (as a wider tensor's slice)."""
    wide = 160 + latent // 2
    cache = torch.randint(0, 256, (rows, wide + pad), generator=g, device="cuda", dtype=torch.uint8)
    at = latent // 2
    key = torch.randn(rows, ROPE, generator=g, device="cuda").to(torch.bfloat16)
    cache[:, at:at + 2 * ROPE] = key.view(torch.uint8)
    cache[:, at + 2 * ROPE:at + 2 * ROPE + 32] = torch.randint(0x18, 0x31, (rows, 32), generator=g, device="cuda",
                                                             dtype=torch.uint8)
    return cache[:, :wide]


def set_value(cache, rows, latent, column, code, scale):
    """Gives value `column` of rows this code, and its block this scale code."""
    at = column // 2
    old = cache[rows, at]
    cache[rows, at] = (old & 0xF0 | code) if column % 2 == 0 else (old & 0x0F | code << 4)
    cache[rows, latent // 2 + 2 * ROPE + column // 16] = scale


def set_key(cache, rows, latent, column, value):
    """Sets a value of rows' key part (column 0 .. 63)."""
    two = torch.tensor([value], device=cache.device).to(torch.bfloat16).view(torch.uint8)
    at = latent // 2 + 2 * column
    cache[rows, at] = two[0]
    cache[rows, at + 1] = two[1]


def attend(query, values, visible, scale, latent):
    """(out, lse, tolerance of out, tolerance of lse), each row from its visible values' rows alone.

    Scores: as in the BF16 form (latent_ref.attend), 2^-16 of sum |q k| and what the
    query loses as FP16: nothing where a value is at least 2^-22 of its row's largest,
    else at most half a step of 2^-24 where the largest is at least 2^8, 2^-33 of it.
    Weights p are rounded to FP16: 2^-11 of themselves, or half a step of 2^-24 where
    the largest is at least 2^8: 2^-25 / 2^8 = 2^-33 of it, and so of their sum at most. The result
    is rounded to BF16 once. 10 % for products of these, 2^-100 for what underflows.
    """
    tokens, heads, _ = query.shape
    out = torch.zeros(tokens, heads, latent, dtype=torch.float64, device=query.device)
    lse = torch.full((tokens, heads), -R.INF, dtype=torch.float64, device=query.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for t, rows in enumerate(visible):
        if rows.numel() == 0:
            continue
        q, keys = query[t].double(), values[rows]
        c = keys[:, :latent]
        s = q @ keys.T * scale
        m = s.amax(1, keepdim=True)
        p = torch.exp(s - m)
        total = p.sum(1, keepdim=True)
        p = p / total
        lse[t] = (m + total.log())[:, 0]
        out[t] = p @ c
        lost = q.abs().amax(1, keepdim=True) * c.abs().sum(1).amax() * 2.0 ** -33
        d = ((q.abs() @ keys.abs().T).amax(1, keepdim=True) * 2.0 ** -16 + lost) * abs(scale)
        tol[t] = 1.1 * (R.U16 * out[t].abs() + (2.0 ** -11 + 2 * d + 2.0 ** -20) * (p @ c.abs())
                        + 2.0 ** -33 * c.abs().sum(0)) + 2.0 ** -100
        tol_lse[t] = d[:, 0] + 2.0 ** -20 * (1 + lse[t].abs())
    return out, lse, tol, tol_lse
