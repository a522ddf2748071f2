"""ctypes mirror of include/latent_bf16.h, latent4.h and page_step.h."""
from __future__ import annotations

import ctypes

_P, _L, _I, _F, _D = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_double


class Append(ctypes.Structure):
    _fields_ = [("cache", _P), ("cache_stride", _L), ("latents", _P), ("latents_stride", _L),
                ("key_rope", _P), ("key_stride", _L), ("positions", _P), ("cos_sin", _P), ("slots", _P),
                ("weight", _P), ("query_rope", _P), ("query_rope_token_stride", _L),
                ("query_rope_head_stride", _L), ("query", _P), ("query_token_stride", _L),
                ("query_head_stride", _L), ("cache_rows", _I), ("tokens", _I), ("latent", _I),
                ("heads", _I), ("max_positions", _I), ("interleaved", _I), ("eps", _F)]


class Attend(ctypes.Structure):
    _fields_ = [("query", _P), ("query_token_stride", _L), ("query_head_stride", _L), ("cache", _P),
                ("cache_stride", _L), ("selected", _P), ("selected_stride", _L), ("valid_len", _P),
                ("block_table", _P), ("out", _P), ("lse", _P), ("workspace", _P), ("workspace_bytes", _L),
                ("cache_rows", _I), ("tokens", _I), ("heads", _I), ("latent", _I), ("k", _I),
                ("width", _I), ("table_stride", _I), ("page_size", _I), ("block_rows", _I),
                ("rows_per_request", _I), ("scale", _F)]


class Append4(ctypes.Structure):
    _fields_ = [*Append._fields_[:-1], ("eps", _D)]


# latent4_attend_t has latent_bf16_attend_t's fields.


class PageStep(ctypes.Structure):
    _fields_ = [("block_table", _P), ("table_stride", _L), ("lengths", _P), ("new_tokens", _P), ("free_pages", _P),
                ("free_count", _P), ("next_lengths", _P), ("next_free_count", _P), ("granted", _P),
                ("positions", _P), ("slots", _P), ("valid_len", _P), ("requests", _I), ("pages", _I),
                ("free_size", _I), ("page_size", _I), ("block_rows", _I), ("rows_per_request", _I),
                ("held", ctypes.c_size_t)]      # an address, 0 for none: the one that may be missing


def declare(lib) -> None:
    """Argument types of the entry points of those headers in a loaded library."""
    for f, args in ((lib.latent_bf16_append, Append), (lib.latent_bf16_attend_selected, Attend),
                    (lib.latent_bf16_attend_paged, Attend), (lib.latent4_append, Append4),
                    (lib.latent4_attend_selected, Attend), (lib.latent4_attend_paged, Attend),
                    (lib.page_step, PageStep)):
        f.argtypes = [ctypes.POINTER(args), _P]
        f.restype = ctypes.c_int
    lib.latent4_rows.argtypes = [_P, _L, _I, _I, _P, _I, _P, _L, _P]
    lib.latent4_rows.restype = ctypes.c_int
    for f in (lib.latent_bf16_attend_workspace, lib.latent4_attend_workspace):
        f.argtypes = [ctypes.POINTER(Attend), _I]
        f.restype = ctypes.c_int64
    for f in (lib.latent_bf16_workspace_bytes, lib.latent4_workspace_bytes):
        f.argtypes = []
        f.restype = ctypes.c_int64
