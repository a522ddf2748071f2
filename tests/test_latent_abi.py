"""The latent-cache operators' C ABI without a GPU: symbols, struct layouts, and
bad arguments refused on the host before touching CUDA."""
import ctypes
import os
import re
import subprocess

import pytest

import exact_bf16_top_gb300 as tk
from exact_bf16_top_gb300._latent_abi import Append, Attend

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "latent_bf16.h")


@pytest.fixture(scope="module")
def lib():
    tk._build.build()
    return tk.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(latent_bf16_\w+)\s*\(", text)))
    assert len(names) == 5
    out = subprocess.run(["nm", "-D", "--defined-only", tk.library_path()], capture_output=True, text=True,
                         check=True).stdout
    for name in names:
        assert re.search(rf"\b{name}\b", out), name
        assert getattr(lib, name) is not None


@pytest.mark.parametrize("mirror,name", [(Append, "latent_bf16_append_t"), (Attend, "latent_bf16_attend_t")])
def test_struct_layouts_match_the_header(tmp_path, mirror, name):
    fields = [f for f, _ in mirror._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "latent_bf16.h"\n'
                   f'int main(void){{printf("%zu", sizeof({name}));'
                   + "".join(f'printf(" %zu", offsetof({name}, {f}));' for f in fields) + 'return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(mirror)] + [getattr(mirror, f).offset for f in fields]


def append_args(**kw):
    a = dict(cache=4096, cache_stride=576, latents=4096, latents_stride=512, key_rope=4096, key_stride=64,
             positions=4096, cos_sin=4096, slots=4096, weight=4096, query_rope=4096, query_rope_token_stride=1024,
             query_rope_head_stride=64, query=4096, query_token_stride=9216, query_head_stride=576, cache_rows=64,
             tokens=2, latent=512, heads=16, max_positions=10, interleaved=1, eps=1e-6)
    a.update(kw)
    return Append(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(cache=None), 1), (dict(latents=None), 1), (dict(key_rope=None), 1), (dict(positions=None), 1),
    (dict(cos_sin=None), 1), (dict(slots=None), 1), (dict(query=None), 1), (dict(query_rope=None), 1),
    (dict(tokens=-1), 1), (dict(tokens=(1 << 27) + 1), 1), (dict(cache_rows=-1), 1), (dict(max_positions=0), 1),
    (dict(heads=0), 1), (dict(heads=257), 1), (dict(latent=500), 4), (dict(latent=0), 4), (dict(latent=640), 4),
    (dict(cache_stride=568), 4), (dict(latents_stride=504), 4), (dict(key_stride=56), 4),
    (dict(query_head_stride=512), 4), (dict(query_token_stride=512), 4), (dict(query_rope_head_stride=-64), 4),
    (dict(cache=4104), 2), (dict(latents=4104), 2), (dict(weight=4098), 2), (dict(cos_sin=4100), 2),
    (dict(positions=4098), 2), (dict(cache_stride=580), 2), (dict(query_rope_token_stride=1028), 2),
    (dict(query=4100), 2),
])
def test_append_refuses(lib, kw, status):
    assert lib.latent_bf16_append(append_args(**kw), None) == status


def attend_args(**kw):
    a = dict(query=4096, query_token_stride=9216, query_head_stride=576, cache=4096, cache_stride=576, selected=4096,
             selected_stride=100, valid_len=4096, block_table=4096, out=4096, lse=4096, workspace=None,
             workspace_bytes=0, cache_rows=64, tokens=2, heads=16, latent=512, k=100, width=100, table_stride=2,
             page_size=64, block_rows=64, rows_per_request=1, scale=0.1)
    a.update(kw)
    return Attend(**a)


COMMON = [
    (dict(query=None), 1), (dict(cache=None), 1), (dict(out=None), 1), (dict(tokens=-1), 1), (dict(cache_rows=-1), 1),
    (dict(heads=0), 1), (dict(heads=257), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1),
    (dict(tokens=1 << 28), 1), (dict(latent=320), 4), (dict(cache_stride=512), 4), (dict(query_head_stride=-576), 4),
    (dict(query=4104), 2), (dict(cache=4104), 2), (dict(out=4104), 2), (dict(lse=4098), 2), (dict(workspace=4104), 2),
    (dict(cache_stride=580), 2), (dict(query_token_stride=9220), 2),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(selected=None), 1), (dict(k=-1), 1), (dict(k=(1 << 30) + 1, selected_stride=1 << 31), 1),
    (dict(selected_stride=99), 4), (dict(selected=4098), 2)])
def test_attend_selected_refuses(lib, kw, status):
    assert lib.latent_bf16_attend_selected(attend_args(**kw), None) == status
    assert lib.latent_bf16_attend_workspace(attend_args(**kw), 0) == -1


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(valid_len=None), 1), (dict(block_table=None), 1), (dict(page_size=48), 1), (dict(page_size=0), 1),
    (dict(block_rows=32), 1), (dict(rows_per_request=0), 1), (dict(table_stride=1), 1), (dict(width=-1), 4),
    (dict(width=(1 << 30) + 1, table_stride=1 << 25), 4), (dict(valid_len=4098), 2), (dict(block_table=4098), 2)])
def test_attend_paged_refuses(lib, kw, status):
    assert lib.latent_bf16_attend_paged(attend_args(**kw), None) == status
    assert lib.latent_bf16_attend_workspace(attend_args(**kw), 1) == -1


def test_no_tokens_is_a_no_op(lib):
    assert lib.latent_bf16_append(append_args(tokens=0, cache=None, latents=None), None) == 0
    assert lib.latent_bf16_attend_selected(attend_args(tokens=0, query=None, out=None), None) == 0
    assert lib.latent_bf16_attend_paged(attend_args(tokens=0, query=None, out=None), None) == 0
    assert lib.latent_bf16_attend_workspace(attend_args(tokens=0, query=None, out=None), 0) == 0
    for f in (lib.latent_bf16_append, lib.latent_bf16_attend_selected, lib.latent_bf16_attend_paged):
        assert f(None, None) == 1


def test_the_names_are_reached_through_the_package():
    for name in ("latent_append", "latent_attend_selected", "latent_attend_paged", "latent_workspace"):
        assert callable(getattr(tk, name))
    with pytest.raises(AttributeError):
        tk.latent_nothing
