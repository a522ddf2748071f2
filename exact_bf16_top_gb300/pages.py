"""A batch's page tables on the GPU: Python binding of ``include/page_step.h``
(argument marshalling only).

``page_step`` gives requests the pages that their new tokens need, takes finished
requests' pages back, and writes every row's position, cache row and valid length:
the block table, ``slots``, ``positions`` and ``valid_len`` that the top-k and the
latent-cache operators take.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

import exact_bf16_top_gb300 as _package

from . import TopkError, load
from ._latent_abi import PageStep as _Args
from .latent import MAX_ROWS, _check_stream, _raw_device, _raw_stream, _refuse

MAX_REQUESTS = 32768
MAX_WIDTH = 1 << 30

_I32 = torch.int32


class PageStep(NamedTuple):
    """What a step gives (int32, on the tables' device): per row (rows_per_request to a request) its position,
    physical cache row (-1: none) and valid length (0: a padded row); per request the tokens it got."""
    positions: torch.Tensor
    slots: torch.Tensor
    valid_len: torch.Tensor
    granted: torch.Tensor


def _vector(t, n: int, dev: int) -> bool:
    return (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is _I32 and t.dim() == 1
            and t.shape[0] == n and t.is_contiguous())


def page_step(block_table, lengths, new_tokens, free_pages, free_count, *, rows_per_request: int = 1,
              page_size: int = 64, block_rows: int | None = None, next_lengths=None, next_free_count=None,
              held=None, stream=None) -> PageStep:
    """Takes a batch's page tables one step further (page_step) -> PageStep.

    block_table: CUDA int32 [requests, pages], request r's first ceil(lengths[r]
    / page_size) entries its pages; lengths: int32 [requests]; new_tokens: int32
    [requests]: tokens that a request gets now (at most rows_per_request), or
    negative for a finished request, whose length becomes 0 and whose pages go
    back; free_pages: int32 [n], of which the first free_count (int32 [1]) are
    the stack of pages that nobody has. The table and the stack are updated in
    place, and so are lengths and free_count unless next_lengths and
    next_free_count (the same shapes) are given for their new values. New pages
    come from the top of the stack downwards, pages that come back lie on it for the
    next step. A request that the table or the stack has no room for gets
    nothing (granted 0) and keeps what it has. block_rows: physical rows per page
    (default page_size). Row r * rows_per_request + j is request r's j-th new
    token: position lengths[r] + j, its slot, valid length position + 1; rows past
    granted[r] are padding (0, -1, 0), which the other operators leave out.

    held: None, or int32 [requests], the pages that each request has, updated in
    place (zeros to begin with will do). It is needed where lengths are lowered
    between steps (drafted tokens that were rejected): a page behind a request's
    last token stays its own, to be used next. Without it a request has what its
    length says, and such a page would be nobody's.
    """
    try:
        dev = block_table.get_device()
        n, pages = block_table.shape
        stride, t1 = block_table.stride()
        (size,), (count,) = free_pages.shape, free_count.shape
        fine = (dev >= 0 and lengths.get_device() == new_tokens.get_device() == dev
                and free_pages.get_device() == free_count.get_device() == dev
                and block_table.dtype is lengths.dtype is new_tokens.dtype is _I32
                and free_pages.dtype is free_count.dtype is _I32 and lengths.shape == new_tokens.shape == (n,)
                and count == 1 and (t1 == 1 or pages <= 1) and lengths.is_contiguous()
                and new_tokens.is_contiguous() and free_pages.is_contiguous())
    except (AttributeError, ValueError):
        fine = False
    if not fine:
        try:
            _refuse(block_table=(block_table, _I32, 2), lengths=(lengths, _I32, 1), new_tokens=(new_tokens, _I32, 1),
                    free_pages=(free_pages, _I32, 1), free_count=(free_count, _I32, 1))
        except ValueError as e:
            if "fit the call" not in str(e):
                raise
            raise ValueError("lengths and new_tokens must have one entry per request, free_count one") from None
    q, page_size = int(rows_per_request), int(page_size)
    if page_size < 1 or page_size & (page_size - 1) or q < 1:
        raise ValueError("page_size must be a power of two and rows_per_request at least 1")
    block_rows = page_size if block_rows is None else int(block_rows)
    if n > MAX_REQUESTS or pages * page_size > MAX_WIDTH:
        raise ValueError(f"at most {MAX_REQUESTS} requests and {MAX_WIDTH} tokens in a request's pages")
    if max(n * pages, n * q, abs(block_rows), page_size, size) > MAX_ROWS:
        raise ValueError("a length or count passes 31 bits")
    if n > 1 and stride < pages:
        raise ValueError("block_table's rows must not overlap")
    if next_lengths is None:
        next_lengths = lengths
    elif not _vector(next_lengths, n, dev):
        raise ValueError("next_lengths must be a contiguous int32 [requests] on the tables' device")
    if next_free_count is None:
        next_free_count = free_count
    elif not _vector(next_free_count, 1, dev):
        raise ValueError("next_free_count must be a contiguous int32 [1] on the tables' device")
    if held is not None and not _vector(held, n, dev):
        raise ValueError("held must be a contiguous int32 [requests] on the tables' device")
    if stream is not None:
        _check_stream(stream, dev)
    if _raw_device() != dev:
        with torch.cuda.device(dev):
            return page_step(block_table, lengths, new_tokens, free_pages, free_count, rows_per_request=q,
                             page_size=page_size, block_rows=block_rows, next_lengths=next_lengths,
                             next_free_count=next_free_count, held=held, stream=stream)
    if stream is not None and stream != torch.cuda.current_stream(dev):
        with torch.cuda.stream(stream):     # new tensors belong to the stream that uses them
            return page_step(block_table, lengths, new_tokens, free_pages, free_count, rows_per_request=q,
                             page_size=page_size, block_rows=block_rows, next_lengths=next_lengths,
                             next_free_count=next_free_count, held=held)
    rows = n * q
    device = block_table.device
    positions, slots = torch.empty(rows, dtype=_I32, device=device), torch.empty(rows, dtype=_I32, device=device)
    valid_len, granted = torch.empty(rows, dtype=_I32, device=device), torch.empty(n, dtype=_I32, device=device)
    args = _Args(block_table.data_ptr(), stride if n > 1 else pages, lengths.data_ptr(), new_tokens.data_ptr(),
                 free_pages.data_ptr(), free_count.data_ptr(), next_lengths.data_ptr(), next_free_count.data_ptr(),
                 granted.data_ptr(), positions.data_ptr(), slots.data_ptr(), valid_len.data_ptr(), n, pages, size,
                 page_size, block_rows, q, 0 if held is None else held.data_ptr())
    status = (_package._lib or load()).page_step(args, _raw_stream(dev))
    if status:
        raise TopkError(status)
    return PageStep(positions, slots, valid_len, granted)
