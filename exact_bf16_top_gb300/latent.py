"""Operators over a paged cache of shared latent rows: Python binding of
``include/latent_bf16.h`` (argument marshalling only, as the top-k's binding).

A cache row holds one token for all heads: ``latent`` values that are key and
value, then 64 rotated values that are key only. ``latent_append`` writes new
tokens' rows; ``latent_attend_selected`` attends over the rows the top-k
selected; ``latent_attend_paged`` over the first tokens of a request's pages.
They have no gradient: where gradients are recorded, tensors that require one
are refused.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

import exact_bf16_top_gb300 as _package

from . import TopkError, load
from ._latent_abi import Append, Attend

ROPE = 64
LATENTS = (128, 256, 384, 512)
MAX_HEADS = 256
MAX_ROWS = 2 ** 31 - 1

_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
# (Plain integers: a step's smallest calls take a few microseconds on the host. A torch without CUDA
# has neither, nor a tensor that gets as far as their use.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


class Form(NamedTuple):
    """How a cache holds its rows, and the entry points that take it."""
    dtype: torch.dtype
    granule: int            # a row's stride is a multiple of this many elements
    columns: dict           # elements of a row by latent
    arguments: type
    append: str
    attend: tuple           # over selected rows, over pages
    workspace: str


BF16 = Form(_BF16, 8, {n: n + ROPE for n in LATENTS}, Append, "latent_bf16_append",
            ("latent_bf16_attend_selected", "latent_bf16_attend_paged"), "latent_bf16_attend_workspace")


def _refuse(**tensors):
    """Raises for the first of name=(tensor, dtype, rank) that does not fit, on the first one's device."""
    dev = None
    for name, (t, dtype, dim) in tensors.items():
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}")
        dev = t.device if dev is None else dev
        if t.device != dev:
            raise ValueError(f"{name} must be on {dev}")
        if t.dim() != dim or (t.shape[-1] > 1 and t.stride(-1) != 1):
            raise ValueError(f"{name} must have {dim} dimension(s) with unit inner stride")
    raise ValueError("tensors do not fit the call")


def _check_no_grad():
    if torch.is_grad_enabled():
        raise ValueError("the latent-cache operators have no gradient: call them under torch.no_grad(), or with "
                         "tensors that do not require one")


def _check_stream(stream, dev: int):
    if stream.device_index != dev:
        raise ValueError(f"stream must be one of cuda:{dev}, where the tensors are")


def _row_stride(rows: int, width: int, stride: int, granule: int = 8) -> int:
    """Row stride of a 2-D tensor; a single row's is immaterial, its width rounded up is given."""
    return stride if rows > 1 else -(-width // granule) * granule


def _head_strides(t) -> tuple[int, int]:
    """Token and head stride of a [tokens, heads, n] tensor (immaterial ones of single rows made plain)."""
    tokens, heads, n = t.shape
    token, head, _ = t.stride()
    if heads == 1:
        head = -(-n // 8) * 8
    return (token if tokens > 1 else max(-(-n // 8) * 8, head * heads)), head


def latent_append(cache, latent, key_rope, positions, cos_sin, slots, *, weight=None, eps: float = 1e-6,
                  interleaved: bool = True, query_rope=None, query=None, stream=None):
    """Writes tokens' rows into the cache (latent_bf16_append) and returns it.

    cache: CUDA bfloat16 [rows, latent + 64], written at ``slots`` (CUDA int32
    [tokens], physical rows, distinct; a token whose slot lies outside the cache,
    e.g. -1, is not written); latent: bfloat16 [tokens, 128 | 256 | 384 | 512]; key_rope:
    bfloat16 [tokens, 64]; positions: int32 [tokens]; cos_sin: float32
    [positions, 64], a position's 32 cosines then 32 sines; weight: None (no
    norm) or bfloat16 [latent], of x * weight / sqrt(mean(x^2) + eps);
    interleaved: rotated pairs are (2 i, 2 i + 1), else (i, i + 32).
    query_rope (bfloat16 [tokens, heads, 64]) and query (bfloat16 [tokens,
    heads, latent + 64]): the same tokens' rotated query parts are written to
    query[..., latent:], which query_rope may be itself; the rest of query is left
    alone. Other overlaps of what is written with what is read are not allowed.
    Rows may be strided: strides multiples of 8, 16-byte aligned.
    """
    return _append(BF16, cache, latent, key_rope, positions, cos_sin, slots, weight, eps, interleaved, query_rope, query,
                   stream)


def latent_attend_selected(query, cache, selected, scale: float, *, latent: int = 512, out=None, lse=False,
                           workspace=None, stream=None):
    """Attention over each token's own list of cache rows: (out, lse).

    query: CUDA bfloat16 [tokens, heads, latent + 64]; cache: bfloat16 [rows,
    latent + 64]; selected: int32 [tokens, k], physical rows as the top-k writes
    them in token mode, in any order (entries outside the cache, e.g. -1, are
    empty places; a block-mode selection's blocks are not rows). out: bfloat16
    [tokens, heads, latent], zero where a token sees nothing; lse: true for the
    float32 [tokens, heads] logarithm of the softmax sum (-inf where a token
    sees nothing), else None is returned for it. workspace: None, or scratch
    from latent_workspace() that no other call uses at the same time.
    """
    return _selected(BF16, query, cache, selected, scale, latent, out, lse, workspace, stream)


def latent_attend_paged(query, cache, valid_len, block_table, scale: float, *, page_size: int = 64,
                        block_rows: int | None = None, rows_per_request: int = 1, width: int | None = None,
                        latent: int = 512, out=None, lse=False, workspace=None, stream=None):
    """Attention over the first valid_len[t] tokens of each request's pages: (out, lse).

    Token t belongs to request t // rows_per_request; valid_len: CUDA int32
    [tokens], clamped to [0, width] (default: the whole table); block_table:
    int32 [requests, pages]; token i of a request is cache row table[i //
    page_size] * block_rows + i % page_size (block_rows: default page_size). A
    chunk of new tokens after n others has valid_len n + 1, n + 2, ...; a padded
    token has 0. Other arguments and results as latent_attend_selected.
    """
    return _paged(BF16, query, cache, valid_len, block_table, scale, page_size, block_rows, rows_per_request, width,
                  latent, out, lse, workspace, stream)


def latent_workspace(device=None):
    """Scratch that is enough for any one attention call at a time on a device (uint8)."""
    return _workspace(device, "latent_bf16_workspace_bytes")


def _workspace(device, function):
    dev = torch.cuda.current_device() if device is None else torch.empty(0, device=device).get_device()
    with torch.cuda.device(dev):
        n = getattr(load(), function)()
    if n <= 0:
        raise RuntimeError("no usable CUDA device")
    return torch.empty(n, dtype=_U8, device=torch.device("cuda", dev))


def _selected(form, query, cache, selected, scale, latent, out, lse, workspace, stream):
    try:
        dev = query.get_device()
        lists, k = selected.shape
        stride, s1 = selected.stride()
        fine = (selected.get_device() == dev and selected.dtype is _I32 and (s1 == 1 or k <= 1))
    except (AttributeError, ValueError):
        fine = False
    if not fine:
        _refuse(query=(query, _BF16, 3), cache=(cache, form.dtype, 2), selected=(selected, _I32, 2))
    if lists != query.shape[0]:
        raise ValueError("selected must have one row per query token")
    if k > MAX_ROWS:
        raise ValueError(f"selected must have at most {MAX_ROWS} entries per row")
    return _attend(form, 0, dev, query, cache, scale, latent, out, lse, workspace, stream,
                   (selected.data_ptr() if k else None, stride if lists > 1 else k, None, None),
                   (k, 0, 0, 1, 1, 1))


def _paged(form, query, cache, valid_len, block_table, scale, page_size, block_rows, rows_per_request, width, latent,
           out, lse, workspace, stream):
    try:
        dev = query.get_device()
        requests, pages = block_table.shape
        stride, t1 = block_table.stride()
        fine = (valid_len.get_device() == block_table.get_device() == dev
                and valid_len.dtype is block_table.dtype is _I32 and valid_len.dim() == 1
                and valid_len.is_contiguous() and (t1 == 1 or pages <= 1))
    except (AttributeError, ValueError):
        fine = False
    if not fine:
        _refuse(query=(query, _BF16, 3), cache=(cache, form.dtype, 2), valid_len=(valid_len, _I32, 1),
                block_table=(block_table, _I32, 2))
    page_size, rows_per_request = int(page_size), int(rows_per_request)
    if page_size < 1 or page_size & (page_size - 1) or rows_per_request < 1:
        raise ValueError("page_size must be a power of two and rows_per_request at least 1")
    tokens = query.shape[0]
    if valid_len.shape[0] != tokens or requests < -(-tokens // rows_per_request):
        raise ValueError("valid_len must have one entry per token, block_table one row per request")
    width = pages * page_size if width is None else int(width)
    if not 0 <= width <= pages * page_size:
        raise ValueError("width exceeds the block table")
    block_rows = page_size if block_rows is None else int(block_rows)
    if max(width, stride, rows_per_request, page_size, abs(block_rows)) > MAX_ROWS:
        raise ValueError("a length, stride or count passes 31 bits")
    return _attend(form, 1, dev, query, cache, scale, latent, out, lse, workspace, stream,
                   (None, 0, valid_len.data_ptr(), block_table.data_ptr()),
                   (0, width, stride if requests > 1 else pages, page_size, block_rows, rows_per_request))


def _attend(form, paged, dev, query, cache, scale, latent, out, lse, workspace, stream, pointers, sizes):
    try:
        tokens, heads, dim = query.shape
        rows, columns = cache.shape
        cache_stride, c1 = cache.stride()
        fine = (dev >= 0 and cache.get_device() == dev and query.dtype is _BF16 and cache.dtype is form.dtype
                and query.stride(2) == 1 and c1 == 1)
    except (AttributeError, ValueError):
        fine = False
    if not fine:
        _refuse(query=(query, _BF16, 3), cache=(cache, form.dtype, 2))
    if rows > MAX_ROWS:
        raise ValueError(f"cache must have at most {MAX_ROWS} rows")
    if form.columns.get(latent) != columns or dim != latent + ROPE:
        raise ValueError(f"latent must be one of {LATENTS}, query rows latent + {ROPE} values, cache rows one of "
                         f"{[*form.columns.values()]} columns")
    if not 1 <= heads <= MAX_HEADS:
        raise ValueError(f"heads must be in [1, {MAX_HEADS}]")
    if query.requires_grad or cache.requires_grad:
        _check_no_grad()
    if stream is not None:
        _check_stream(stream, dev)
    if _raw_device() != dev:
        with torch.cuda.device(dev):
            return _attend(form, paged, dev, query, cache, scale, latent, out, lse, workspace, stream, pointers,
                           sizes)
    if stream is not None and stream != torch.cuda.current_stream(dev):
        with torch.cuda.stream(stream):     # new tensors belong to the stream that uses them
            return _attend(form, paged, dev, query, cache, scale, latent, out, lse, workspace, None, pointers, sizes)
    device = query.device
    if out is None:
        out = torch.empty((tokens, heads, latent), dtype=_BF16, device=device)
    elif not (out.dtype is _BF16 and out.device == device and out.shape == (tokens, heads, latent)
              and out.is_contiguous()):
        raise ValueError("out must be a contiguous bfloat16 [tokens, heads, latent] on the query's device")
    elif out.requires_grad:
        _check_no_grad()
    if not isinstance(lse, torch.Tensor):
        lse = torch.empty((tokens, heads), dtype=_F32, device=device) if lse else None
    elif not (lse.dtype is _F32 and lse.device == device and lse.shape == (tokens, heads) and lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [tokens, heads] on the query's device")
    elif lse.requires_grad:
        _check_no_grad()
    if workspace is not None and not (workspace.dtype is _U8 and workspace.device == device
                                      and workspace.is_contiguous()):
        raise ValueError("workspace must be a uint8 tensor from latent_workspace() on the query's device")
    lse_ptr = None if lse is None else lse.data_ptr()
    if tokens:
        args = Attend(query.data_ptr(), *_head_strides(query), cache.data_ptr(),
                      _row_stride(rows, columns, cache_stride, form.granule), *pointers, out.data_ptr(), lse_ptr,
                      None, 0, rows, tokens, heads, latent, *sizes, scale)
        lib = _package._lib or load()
        if workspace is None:
            n = getattr(lib, form.workspace)(args, paged)
            if n > 0:
                workspace = torch.empty(n, dtype=_U8, device=device)
        if workspace is not None:
            args.workspace, args.workspace_bytes = workspace.data_ptr(), workspace.numel()
        status = getattr(lib, form.attend[paged])(args, _raw_stream(dev))
        if status:
            raise TopkError(status)
    return out, lse


def _append(form, cache, latent, key_rope, positions, cos_sin, slots, weight, eps, interleaved, query_rope, query,
            stream):
    try:
        dev = cache.get_device()
        rows, columns = cache.shape
        cache_stride, c1 = cache.stride()
        tokens, width = latent.shape
        latent_stride, l1 = latent.stride()
        key_stride, k1 = key_rope.stride()
        fine = (dev >= 0 and latent.get_device() == key_rope.get_device() == positions.get_device() == dev
                and cos_sin.get_device() == slots.get_device() == dev
                and cache.dtype is form.dtype and latent.dtype is key_rope.dtype is _BF16
                and positions.dtype is slots.dtype is _I32 and cos_sin.dtype is _F32
                and c1 == l1 == k1 == 1 and positions.is_contiguous() and slots.is_contiguous()
                and positions.dim() == slots.dim() == 1 and cos_sin.dim() == 2)
    except (AttributeError, ValueError):
        fine = False
    if not fine:
        _refuse(cache=(cache, form.dtype, 2), latent=(latent, _BF16, 2), key_rope=(key_rope, _BF16, 2),
                positions=(positions, _I32, 1), cos_sin=(cos_sin, _F32, 2), slots=(slots, _I32, 1))
    if rows > MAX_ROWS or tokens > MAX_ROWS:
        raise ValueError(f"at most {MAX_ROWS} cache rows and tokens")
    if form.columns.get(width) != columns:
        raise ValueError(f"latent must have one of {LATENTS} columns and cache {[*form.columns.values()]}")
    dim = width + ROPE
    if key_rope.shape != (tokens, ROPE) or positions.shape[0] != tokens or slots.shape[0] != tokens:
        raise ValueError("key_rope, positions and slots must have one row per token (key_rope of 64)")
    positions_known, angles = cos_sin.shape
    if angles != ROPE or positions_known < 1 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be contiguous [positions, 64]")
    weight_ptr = None
    if weight is not None:
        if not (isinstance(weight, torch.Tensor) and weight.get_device() == dev and weight.dtype is _BF16
                and weight.dim() == 1 and weight.is_contiguous()):
            _refuse(cache=(cache, form.dtype, 2), weight=(weight, _BF16, 1))
        if weight.shape[0] != width:
            raise ValueError("weight must have one entry per latent column")
        weight_ptr = weight.data_ptr()
    if (query is None) != (query_rope is None):
        raise ValueError("query and query_rope come together")
    if query is None:
        heads, r, q = 0, (None, 0, 0), (None, 0, 0)
    else:
        if not (isinstance(query, torch.Tensor) and isinstance(query_rope, torch.Tensor)
                and query.get_device() == query_rope.get_device() == dev
                and query.dtype is query_rope.dtype is _BF16 and query.dim() == query_rope.dim() == 3
                and query.stride(2) == query_rope.stride(2) == 1):
            _refuse(cache=(cache, form.dtype, 2), query=(query, _BF16, 3), query_rope=(query_rope, _BF16, 3))
        heads = query.shape[1]
        if query.shape != (tokens, heads, dim) or query_rope.shape != (tokens, heads, ROPE):
            raise ValueError("query must be [tokens, heads, latent + 64] and query_rope [tokens, heads, 64]")
        if not 1 <= heads <= MAX_HEADS:
            raise ValueError(f"heads must be in [1, {MAX_HEADS}]")
        r = (query_rope.data_ptr(), *_head_strides(query_rope))
        q = (query.data_ptr(), *_head_strides(query))
    args = form.arguments(cache.data_ptr(), _row_stride(rows, columns, cache_stride, form.granule), latent.data_ptr(),
                          _row_stride(tokens, width, latent_stride), key_rope.data_ptr(),
                          _row_stride(tokens, ROPE, key_stride), positions.data_ptr(), cos_sin.data_ptr(),
                          slots.data_ptr(), weight_ptr, *r, *q, rows, tokens, width, heads, positions_known,
                          1 if interleaved else 0, eps)
    if (cache.requires_grad or latent.requires_grad or key_rope.requires_grad or cos_sin.requires_grad
            or (weight is not None and weight.requires_grad)
            or (query is not None and (query.requires_grad or query_rope.requires_grad))):
        _check_no_grad()
    if stream is not None:
        _check_stream(stream, dev)
    function = getattr(_package._lib or load(), form.append)
    handle = _raw_stream(dev) if stream is None else stream.cuda_stream
    if _raw_device() == dev:
        status = function(args, handle)
    else:
        with torch.cuda.device(dev):
            status = function(args, handle)
    if status:
        raise TopkError(status)
    return cache
