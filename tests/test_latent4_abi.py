"""The 4-bit latent cache's and the page tables' C ABI without a GPU: symbols, struct
layouts, and bad arguments refused on the host before touching CUDA."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

import exact_bf16_top_gb300 as tk
from exact_bf16_top_gb300._latent_abi import Append4, Attend, PageStep

INCLUDE = os.path.join(tk._build.ROOT, "include")


@pytest.fixture(scope="module")
def lib():
    tk._build.build()
    return tk.load()


@pytest.mark.parametrize("header,prefix,count", [("latent4.h", "latent4_", 6), ("page_step.h", "page_step", 1)])
def test_every_declared_symbol_is_exported(lib, header, prefix, count):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, header)).read(), flags=re.S)
    names = sorted(set(re.findall(rf"\b({prefix}\w*)\s*\(", text)))
    assert len(names) == count
    out = subprocess.run(["nm", "-D", "--defined-only", tk.library_path()], capture_output=True, text=True,
                         check=True).stdout
    for name in names:
        assert re.search(rf"\b{name}\b", out), name
        assert getattr(lib, name) is not None


@pytest.mark.parametrize("mirror,name,header", [(Append4, "latent4_append_t", "latent4.h"),
                                                (Attend, "latent4_attend_t", "latent4.h"),
                                                (PageStep, "page_step_t", "page_step.h")])
def test_struct_layouts_match_the_header(tmp_path, mirror, name, header):
    fields = [f for f, _ in mirror._fields_]
    src = tmp_path / "layout.c"
    src.write_text(f'#include <stddef.h>\n#include <stdio.h>\n#include "{header}"\n'
                   f'int main(void){{printf("%zu", sizeof({name}));'
                   + "".join(f'printf(" %zu", offsetof({name}, {f}));' for f in fields) + 'return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", INCLUDE, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(mirror)] + [getattr(mirror, f).offset for f in fields]


def append_args(**kw):
    a = dict(cache=4096, cache_stride=416, latents=4096, latents_stride=512, key_rope=4096, key_stride=64,
             positions=4096, cos_sin=4096, slots=4096, weight=4096, query_rope=4096, query_rope_token_stride=1024,
             query_rope_head_stride=64, query=4096, query_token_stride=9216, query_head_stride=576, cache_rows=64,
             tokens=2, latent=512, heads=16, max_positions=10, interleaved=1, eps=1e-6)
    a.update(kw)
    return Append4(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(cache=None), 1), (dict(latents=None), 1), (dict(slots=None), 1), (dict(query=None), 1),
    (dict(tokens=-1), 1), (dict(tokens=(1 << 27) + 1), 1), (dict(cache_rows=-1), 1), (dict(max_positions=0), 1),
    (dict(heads=257), 1), (dict(latent=500), 4), (dict(latent=640), 4), (dict(cache_stride=384), 4),
    (dict(latents_stride=504), 4), (dict(query_head_stride=512), 4), (dict(cache=4112), 2), (dict(cache=4100), 2),
    (dict(cache_stride=424), 2), (dict(cache_stride=432), 2), (dict(latents=4104), 2), (dict(latents_stride=516), 2),
    (dict(weight=4098), 2)])
def test_append_refuses(lib, kw, status):
    assert lib.latent4_append(append_args(**kw), None) == status


def attend_args(**kw):
    a = dict(query=4096, query_token_stride=9216, query_head_stride=576, cache=4096, cache_stride=416, selected=4096,
             selected_stride=100, valid_len=4096, block_table=4096, out=4096, lse=4096, workspace=None,
             workspace_bytes=0, cache_rows=64, tokens=2, heads=16, latent=512, k=100, width=100, table_stride=2,
             page_size=64, block_rows=64, rows_per_request=1, scale=0.1)
    a.update(kw)
    return Attend(**a)


@pytest.mark.parametrize("paged", [0, 1])
@pytest.mark.parametrize("kw,status", [
    (dict(query=None), 1), (dict(cache=None), 1), (dict(out=None), 1), (dict(tokens=-1), 1), (dict(cache_rows=-1), 1),
    (dict(heads=0), 1), (dict(heads=257), 1), (dict(scale=float("inf")), 1), (dict(tokens=1 << 28), 1),
    (dict(latent=320), 4), (dict(cache_stride=384), 4), (dict(query_head_stride=-576), 4), (dict(query=4104), 2),
    (dict(cache=4112), 2), (dict(cache_stride=432), 2), (dict(out=4104), 2), (dict(workspace=4104), 2)])
def test_attend_refuses(lib, paged, kw, status):
    f = lib.latent4_attend_paged if paged else lib.latent4_attend_selected
    assert f(attend_args(**kw), None) == status
    assert lib.latent4_attend_workspace(attend_args(**kw), paged) == -1


@pytest.mark.parametrize("args,status", [
    ((None, 416, 9, 512, 4096, 3, 4096, 576), 1), ((4096, 416, 9, 512, None, 3, 4096, 576), 1),
    ((4096, 416, 9, 512, 4096, 3, None, 576), 1), ((4096, 416, -1, 512, 4096, 3, 4096, 576), 1),
    ((4096, 416, 9, 512, 4096, -3, 4096, 576), 1), ((4096, 416, 9, 500, 4096, 3, 4096, 576), 4),
    ((4096, 384, 9, 512, 4096, 3, 4096, 576), 4), ((4096, 416, 9, 512, 4096, 3, 4096, 568), 4),
    ((4112, 416, 9, 512, 4096, 3, 4096, 576), 2), ((4096, 424, 9, 512, 4096, 3, 4096, 576), 2),
    ((4096, 416, 9, 512, 4098, 3, 4096, 576), 2), ((4096, 416, 9, 512, 4096, 3, 4104, 576), 2),
    ((4096, 416, 9, 512, 4096, 3, 4096, 580), 2), ((None, 0, 0, 512, None, 0, None, 0), 0)])
def test_rows_refuses(lib, args, status):
    assert lib.latent4_rows(*args, None) == status


def step_args(**kw):
    a = dict(block_table=4096, table_stride=8, lengths=4096, new_tokens=4096, free_pages=4096, free_count=4096,
             next_lengths=4096, next_free_count=4096, granted=4096, positions=4096, slots=4096, valid_len=4096,
             requests=4, pages=8, free_size=10, page_size=64, block_rows=64, rows_per_request=2)
    a.update(kw)
    return PageStep(**a)


POINTERS = [f for f, t in PageStep._fields_ if t is ctypes.c_void_p]


@pytest.mark.parametrize("kw,status", [(dict([(f, None)]), 1) for f in POINTERS] + [
    (dict([(f, 4098)]), 2) for f in POINTERS] + [
    (dict(requests=-1), 1), (dict(requests=32769), 1), (dict(pages=-1), 1), (dict(free_size=-1), 1),
    (dict(page_size=0), 1), (dict(page_size=48), 1), (dict(block_rows=32), 1), (dict(rows_per_request=0), 1),
    (dict(table_stride=7), 1), (dict(rows_per_request=1 << 30), 1), (dict(requests=32768, pages=65536, table_stride=65536, page_size=1), 1),
    (dict(page_size=1 << 28, block_rows=1 << 28), 4)])
def test_step_refuses(lib, kw, status):
    assert lib.page_step(step_args(**kw), None) == status


def test_step_held_may_be_missing_but_not_misaligned(lib):
    assert PageStep().held == 0
    assert lib.page_step(step_args(held=4098), None) == 2
    assert lib.page_step(step_args(held=4096, lengths=None), None) == 1


def test_nothing_to_do_and_no_arguments(lib):
    assert lib.latent4_append(append_args(tokens=0, cache=None, latents=None), None) == 0
    assert lib.latent4_attend_selected(attend_args(tokens=0, query=None, out=None), None) == 0
    assert lib.latent4_attend_paged(attend_args(tokens=0, query=None, out=None), None) == 0
    assert lib.latent4_attend_workspace(attend_args(tokens=0, query=None, out=None), 0) == 0
    for f in (lib.latent4_append, lib.latent4_attend_selected, lib.latent4_attend_paged, lib.page_step):
        assert f(None, None) == 1


def test_row_bytes():
    src = "#include <stdio.h>\n#include \"latent4.h\"\nint main(void){int v;for(v=128;v<=512;v+=128)printf(\"%d \","
    src += "LATENT4_ROW_BYTES(v));return 0;}"
    exe = "/tmp/latent4_row_bytes"
    subprocess.run(["gcc", "-std=c99", "-I", INCLUDE, "-x", "c", "-", "-o", exe], input=src, text=True, check=True)
    got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == [tk.latent4_row_bytes(v) for v in (128, 256, 384, 512)] == [224, 288, 352, 416]


def test_the_names_are_reached_through_the_package():
    for name in ("latent4_append", "latent4_rows", "latent4_attend_selected", "latent4_attend_paged",
                 "latent4_row_bytes", "latent4_workspace", "page_step"):
        assert callable(getattr(tk, name))


def test_a_torch_without_cuda_gets_the_refusal():
    code = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import exact_bf16_top_gb300 as tk
a = torch.zeros(2, 16, 576, dtype=torch.bfloat16)
c = torch.zeros(64, 416, dtype=torch.uint8)
i = torch.zeros(2, 4, dtype=torch.int32)
for call in (lambda: tk.latent4_attend_selected(a, c, i, 0.1), lambda: tk.latent4_attend_paged(a, c, i[:, 0], i, 0.1),
             lambda: tk.latent4_append(c, a[:, 0, :512], a[:, 0, 512:], i[:, 0], c.float(), i[:, 0]),
             lambda: tk.latent4_rows(c, i[:, 0]), lambda: tk.page_step(i, i[:, 0], i[:, 0], i[:, 0], i[0, :1])):
    try:
        call()
    except TypeError as e:
        assert "CUDA tensor" in str(e), e
    else:
        raise AssertionError("not refused")
"""
    subprocess.run([sys.executable, "-c", code], cwd=tk._build.ROOT, check=True)
