"""ctypes mirror of include/latent_bf16.h."""
from __future__ import annotations

import ctypes

_P, _L, _I, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


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


def declare(lib) -> None:
    """Argument types of the latent entry points of a loaded library."""
    lib.latent_bf16_append.argtypes = [ctypes.POINTER(Append), _P]
    lib.latent_bf16_attend_selected.argtypes = [ctypes.POINTER(Attend), _P]
    lib.latent_bf16_attend_paged.argtypes = [ctypes.POINTER(Attend), _P]
    for f in (lib.latent_bf16_append, lib.latent_bf16_attend_selected, lib.latent_bf16_attend_paged):
        f.restype = ctypes.c_int
    lib.latent_bf16_attend_workspace.argtypes = [ctypes.POINTER(Attend), ctypes.c_int32]
    lib.latent_bf16_attend_workspace.restype = ctypes.c_int64
    lib.latent_bf16_workspace_bytes.argtypes = []
    lib.latent_bf16_workspace_bytes.restype = ctypes.c_int64
