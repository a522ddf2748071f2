"""Operators over a paged cache of latent rows in 4 bits: Python binding of
``include/latent4.h``, with the arguments of ``latent.py``'s.

A cache row is uint8 [latent4_row_bytes(latent)]: latent / 2 bytes of codes
(e2m1, the even value in the low half), 64 BF16 key values, 32 scales (e4m3, one
per 16 values). ``latent4_append`` writes new tokens' rows, ``latent4_rows``
reads rows back, ``latent4_attend_selected`` and ``latent4_attend_paged`` attend
over them.
"""
from __future__ import annotations

import torch

import exact_bf16_top_gb300 as _package

from . import TopkError, load
from ._latent_abi import Append4
from .latent import (_BF16, _I32, _U8, LATENTS, MAX_ROWS, ROPE, Form, _append, _check_no_grad, _check_stream, _paged,
                     _raw_device, _raw_stream, _refuse, _row_stride, _selected, _workspace)


def latent4_row_bytes(latent: int) -> int:
    """Bytes of a cache row of ``latent`` (128, 256, 384 or 512) values."""
    if latent not in LATENTS:
        raise ValueError(f"latent must be one of {LATENTS}")
    return 160 + latent // 2


FP4 = Form(_U8, 32, {n: 160 + n // 2 for n in LATENTS}, Append4, "latent4_append",
           ("latent4_attend_selected", "latent4_attend_paged"), "latent4_attend_workspace")


def latent4_append(cache, latent, key_rope, positions, cos_sin, slots, *, weight=None, eps: float = 1e-6,
                   interleaved: bool = True, query_rope=None, query=None, stream=None):
    """Writes tokens' rows into the 4-bit cache (latent4_append) and returns it.

    cache: CUDA uint8 [rows, latent4_row_bytes(latent)], 32-byte aligned, a
    row's stride a multiple of 32. Everything else as latent_append; latent
    values are rounded to 4 bits once, from the norm as exact arithmetic has it
    (sixteen values of which one is not finite read back as NaN).
    """
    return _append(FP4, cache, latent, key_rope, positions, cos_sin, slots, weight, eps, interleaved, query_rope, query,
                   stream)


def latent4_rows(cache, rows, *, latent: int = 512, out=None, stream=None):
    """Cache rows as bfloat16 [n, latent + 64], exactly (latent4_rows).

    rows: CUDA int32 [n], physical rows; zeros for one outside the cache (-1).
    out: bfloat16 [n, latent + 64] with unit inner stride, 16-byte aligned rows.
    """
    try:
        dev = cache.get_device()
        cached, columns = cache.shape
        cache_stride, c1 = cache.stride()
        count = rows.shape[0]
        fine = (dev >= 0 and rows.get_device() == dev and cache.dtype is _U8 and rows.dtype is _I32 and c1 == 1
                and rows.dim() == 1 and rows.is_contiguous())
    except (AttributeError, ValueError, IndexError):
        fine = False
    if not fine:
        _refuse(cache=(cache, _U8, 2), rows=(rows, _I32, 1))
    if FP4.columns.get(latent) != columns:
        raise ValueError(f"latent must be one of {LATENTS}, cache rows one of {[*FP4.columns.values()]} columns")
    if cached > MAX_ROWS or count > MAX_ROWS:
        raise ValueError(f"at most {MAX_ROWS} rows")
    if stream is not None:
        _check_stream(stream, dev)
    if _raw_device() != dev:
        with torch.cuda.device(dev):
            return latent4_rows(cache, rows, latent=latent, out=out, stream=stream)
    if stream is not None and stream != torch.cuda.current_stream(dev):
        with torch.cuda.stream(stream):     # a new tensor belongs to the stream that uses it
            return latent4_rows(cache, rows, latent=latent, out=out)
    width = latent + ROPE
    if out is None:
        out = torch.empty((count, width), dtype=_BF16, device=cache.device)
    elif not (isinstance(out, torch.Tensor) and out.dtype is _BF16 and out.get_device() == dev
              and out.shape == (count, width) and out.stride(1) == 1):
        raise ValueError("out must be a bfloat16 [rows, latent + 64] with unit inner stride on the cache's device")
    elif out.requires_grad:
        _check_no_grad()
    if count:
        status = (_package._lib or load()).latent4_rows(
            cache.data_ptr(), _row_stride(cached, columns, cache_stride, 32), cached, latent, rows.data_ptr(), count,
            out.data_ptr(), _row_stride(count, width, out.stride(0)), _raw_stream(dev))
        if status:
            raise TopkError(status)
    return out


def latent4_attend_selected(query, cache, selected, scale: float, *, latent: int = 512, out=None, lse=False,
                            workspace=None, stream=None):
    """Attention over each token's own list of 4-bit cache rows: (out, lse).

    cache: CUDA uint8 [rows, latent4_row_bytes(latent)], as latent4_append writes
    it. Everything else as latent_attend_selected (workspace: from
    latent4_workspace()).
    """
    return _selected(FP4, query, cache, selected, scale, latent, out, lse, workspace, stream)


def latent4_attend_paged(query, cache, valid_len, block_table, scale: float, *, page_size: int = 64,
                         block_rows: int | None = None, rows_per_request: int = 1, width: int | None = None,
                         latent: int = 512, out=None, lse=False, workspace=None, stream=None):
    """Attention over the first valid_len[t] tokens of each request's pages of 4-bit rows: (out, lse).

    cache: CUDA uint8 [rows, latent4_row_bytes(latent)], as latent4_append writes
    it. Everything else as latent_attend_paged (workspace: from
    latent4_workspace()).
    """
    return _paged(FP4, query, cache, valid_len, block_table, scale, page_size, block_rows, rows_per_request, width,
                  latent, out, lse, workspace, stream)


def latent4_workspace(device=None):
    """Scratch that is enough for any one 4-bit attention call at a time on a device (uint8)."""
    return _workspace(device, "latent4_workspace_bytes")
