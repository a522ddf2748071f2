"""Operators over a paged cache of shared latent rows: Python binding of
``include/latent_bf16.h`` (argument marshalling only, as the top-k's binding).

A cache row holds one token for all heads: ``latent`` values that are key and
value, then 64 rotated values that are key only. ``latent_append`` writes new
tokens' rows; ``latent_attend_selected`` attends over the rows the top-k
selected; ``latent_attend_paged`` over the first tokens of a request's pages.
"""
from __future__ import annotations

import torch

from ._latent_abi import Append, Attend

ROPE = 64
LATENTS = (128, 256, 384, 512)
MAX_HEADS = 256


def _tensor(t, name: str, dtype, dim: int, device=None):
    """Checks one argument: a CUDA tensor of this type and rank with unit inner stride, on `device`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dim() != dim or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must have {dim} dimension(s) with unit inner stride")


def _row_stride(t) -> int:
    """Row stride of a 2-D tensor; a single row's is immaterial, its width rounded up is given."""
    return t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // 8) * 8


def _head_strides(t) -> tuple[int, int]:
    """Token and head stride of a [tokens, heads, n] tensor (immaterial ones of single rows made plain)."""
    n = -(-t.shape[2] // 8) * 8
    head = t.stride(1) if t.shape[1] > 1 else n
    return (t.stride(0) if t.shape[0] > 1 else max(n, head * t.shape[1])), head


def _launch(function, args, device, stream):
    from . import _check
    if stream is None:
        stream = torch.cuda.current_stream(device)
    if torch.cuda.current_device() == device.index:
        status = function(args, stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            status = function(args, stream.cuda_stream)
    _check(status)


def latent_append(cache, latent, key_rope, positions, cos_sin, slots, *, weight=None, eps: float = 1e-6,
                  interleaved: bool = True, query_rope=None, query=None, stream=None):
    """Writes tokens' rows into the cache (latent_bf16_append) and returns it.

    cache: CUDA bfloat16 [rows, latent + 64], written at ``slots`` (CUDA int32
    [tokens], physical rows; a token whose slot lies outside the cache, e.g. -1,
    is not written); latent: bfloat16 [tokens, 128 | 256 | 384 | 512]; key_rope:
    bfloat16 [tokens, 64]; positions: int32 [tokens]; cos_sin: float32
    [positions, 64], a position's 32 cosines then 32 sines; weight: None (no
    norm) or bfloat16 [latent], of x * weight / sqrt(mean(x^2) + eps);
    interleaved: rotated pairs are (2 i, 2 i + 1), else (i, i + 32).
    query_rope (bfloat16 [tokens, heads, 64]) and query (bfloat16 [tokens,
    heads, latent + 64]): the same tokens' rotated query parts are written to
    query[..., latent:]; the rest of query is left alone.
    Rows may be strided: strides multiples of 8, 16-byte aligned.
    """
    from . import load
    bf16, i32 = torch.bfloat16, torch.int32
    _tensor(cache, "cache", bf16, 2)
    dev = cache.device
    _tensor(latent, "latent", bf16, 2, dev)
    _tensor(key_rope, "key_rope", bf16, 2, dev)
    _tensor(positions, "positions", i32, 1, dev)
    _tensor(cos_sin, "cos_sin", torch.float32, 2, dev)
    _tensor(slots, "slots", i32, 1, dev)
    tokens, width = latent.shape
    if width not in LATENTS or cache.shape[1] != width + ROPE:
        raise ValueError(f"latent must have one of {LATENTS} columns and cache {ROPE} more")
    if key_rope.shape != (tokens, ROPE) or positions.shape[0] != tokens or slots.shape[0] != tokens:
        raise ValueError("key_rope, positions and slots must have one row per token (key_rope of 64)")
    if cos_sin.shape[1] != ROPE or cos_sin.shape[0] < 1 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be contiguous [positions, 64]")
    if weight is not None:
        _tensor(weight, "weight", bf16, 1, dev)
        if weight.shape[0] != width:
            raise ValueError("weight must have one entry per latent column")
    if (query is None) != (query_rope is None):
        raise ValueError("query and query_rope come together")
    heads, q, r = 0, (0, 0), (0, 0)
    if query is not None:
        _tensor(query, "query", bf16, 3, dev)
        _tensor(query_rope, "query_rope", bf16, 3, dev)
        heads = query.shape[1]
        if query.shape != (tokens, heads, width + ROPE) or query_rope.shape != (tokens, heads, ROPE):
            raise ValueError("query must be [tokens, heads, latent + 64] and query_rope [tokens, heads, 64]")
        if not 1 <= heads <= MAX_HEADS:
            raise ValueError(f"heads must be in [1, {MAX_HEADS}]")
        q, r = _head_strides(query), _head_strides(query_rope)
    args = Append(cache.data_ptr(), _row_stride(cache), latent.data_ptr(), _row_stride(latent),
                   key_rope.data_ptr(), _row_stride(key_rope), positions.data_ptr(), cos_sin.data_ptr(),
                   slots.data_ptr(), None if weight is None else weight.data_ptr(),
                   None if query is None else query_rope.data_ptr(), r[0], r[1],
                   None if query is None else query.data_ptr(), q[0], q[1], cache.shape[0], tokens, width,
                   heads, cos_sin.shape[0], 1 if interleaved else 0, eps)
    _launch(load().latent_bf16_append, args, dev, stream)
    return cache


def latent_attend_selected(query, cache, selected, scale: float, *, latent: int = 512, out=None, lse=False,
                           workspace=None, stream=None):
    """Attention over each token's own list of cache rows: (out, lse).

    query: CUDA bfloat16 [tokens, heads, latent + 64]; cache: bfloat16 [rows,
    latent + 64]; selected: int32 [tokens, k], physical rows as the top-k writes
    them (entries outside the cache, e.g. -1, are empty places). out: bfloat16
    [tokens, heads, latent], zero where a token sees nothing; lse: True for the
    float32 [tokens, heads] logarithm of the softmax sum (-inf where a token
    sees nothing), else None is returned for it. workspace: None, or scratch
    from latent_workspace() that no other call uses at the same time.
    """
    _tensor(selected, "selected", torch.int32, 2)
    if selected.shape[0] != query.shape[0]:
        raise ValueError("selected must have one row per query token")
    k = selected.shape[1]
    stride = selected.stride(0) if selected.shape[0] > 1 else k
    return _attend("latent_bf16_attend_selected", query, cache, scale, latent, out, lse, workspace, stream,
                   (selected,), (selected.data_ptr() if k else None, stride, None, None),
                   (k, 0, 0, 1, 1, 1))


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
    _tensor(valid_len, "valid_len", torch.int32, 1)
    _tensor(block_table, "block_table", torch.int32, 2)
    page_size, rows_per_request = int(page_size), int(rows_per_request)
    if page_size < 1 or page_size & (page_size - 1) or rows_per_request < 1:
        raise ValueError("page_size must be a power of two and rows_per_request at least 1")
    tokens, (requests, pages) = query.shape[0], block_table.shape
    if valid_len.shape[0] != tokens or requests < -(-tokens // rows_per_request):
        raise ValueError("valid_len must have one entry per token, block_table one row per request")
    width = pages * page_size if width is None else int(width)
    if not 0 <= width <= pages * page_size:
        raise ValueError("width exceeds the block table")
    stride = block_table.stride(0) if requests > 1 else pages
    return _attend("latent_bf16_attend_paged", query, cache, scale, latent, out, lse, workspace, stream,
                   (valid_len, block_table), (None, 0, valid_len.data_ptr(), block_table.data_ptr()),
                   (0, width, stride, page_size, page_size if block_rows is None else int(block_rows),
                    rows_per_request))


def latent_workspace(device=None):
    """Scratch for one attention call at a time on a device (uint8)."""
    from . import load
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        n = load().latent_bf16_workspace_bytes()
        if n <= 0:
            raise RuntimeError("no usable CUDA device")
        return torch.empty(n, dtype=torch.uint8, device=device)


_workspace_bytes: dict[int, int] = {}


def _attend(name, query, cache, scale, latent, out, lse, workspace, stream, others, pointers, sizes):
    from . import load
    bf16 = torch.bfloat16
    _tensor(query, "query", bf16, 3)
    dev = query.device
    _tensor(cache, "cache", bf16, 2, dev)
    for t in others:
        if t.device != dev:
            raise ValueError(f"all tensors must be on {dev}")
    tokens, heads, dim = query.shape
    if latent not in LATENTS or dim != latent + ROPE or cache.shape[1] != dim:
        raise ValueError(f"latent must be one of {LATENTS}, query and cache rows latent + {ROPE} values")
    if not 1 <= heads <= MAX_HEADS:
        raise ValueError(f"heads must be in [1, {MAX_HEADS}]")
    if stream is not None:
        # Allocated on the stream that uses them.
        with torch.cuda.stream(stream):
            out, lse, workspace = _outputs(out, lse, workspace, dev, tokens, heads, latent)
    else:
        out, lse, workspace = _outputs(out, lse, workspace, dev, tokens, heads, latent)
    if tokens == 0:
        return out, lse
    q = _head_strides(query)
    args = Attend(query.data_ptr(), q[0], q[1], cache.data_ptr(), _row_stride(cache), *pointers,
                   out.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr(),
                   workspace.numel(), cache.shape[0], tokens, heads, latent, *sizes, scale)
    _launch(getattr(load(), name), args, dev, stream)
    return out, lse


def _outputs(out, lse, workspace, dev, tokens, heads, latent):
    """The caller's tensors, checked, or new ones."""
    if out is None:
        out = torch.empty((tokens, heads, latent), dtype=torch.bfloat16, device=dev)
    elif not (out.dtype == torch.bfloat16 and out.device == dev and out.shape == (tokens, heads, latent)
              and out.is_contiguous()):
        raise ValueError("out must be a contiguous bfloat16 [tokens, heads, latent] on the query's device")
    if isinstance(lse, torch.Tensor):
        if not (lse.dtype == torch.float32 and lse.device == dev and lse.shape == (tokens, heads)
                and lse.is_contiguous()):
            raise ValueError("lse must be a contiguous float32 [tokens, heads] on the query's device")
    else:
        lse = torch.empty((tokens, heads), dtype=torch.float32, device=dev) if lse else None
    if workspace is None:
        n = _workspace_bytes.get(dev.index)
        if n is None:
            workspace = latent_workspace(dev)
            _workspace_bytes[dev.index] = workspace.numel()
        else:
            workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    elif not (workspace.dtype == torch.uint8 and workspace.device == dev and workspace.is_contiguous()):
        raise ValueError("workspace must be a uint8 tensor from latent_workspace() on the query's device")
    return out, lse, workspace
