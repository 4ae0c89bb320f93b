"""Host-side checks of the row-format, attention and shared-page calls that
need no GPU: null contexts and calls, sizes, the call structs' layout, and the
binding's checks of tensors."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

from hierarchical_sparse_kv_resolve_amd import kvr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_row_layout():
    assert kvr.row_layout("bf16", 512, 64) == kvr.row_layout("f16", 512, 64) == 1152
    assert kvr.row_layout("fp8", 512, 64) == 656
    assert kvr.row_layout("fp8", 512, 0) == 528
    assert kvr.row_layout("fp8", 256, 64) == 256 + 16 + 128  # two scales and their padding
    assert kvr.row_layout("bf16", 256, 0) == 512
    for fmt, d_v, d_rope in (("bf16", 384, 64), ("fp8", 512, 32), ("f16", 0, 64), ("fp8", 512, -64)):
        with pytest.raises(kvr.KvrError, match="d_v is 256 or 512"):
            kvr.row_layout(fmt, d_v, d_rope)
    with pytest.raises(ValueError, match="unknown row format"):
        kvr.row_layout("int8", 512, 64)
    assert kvr.lib().kvr_row_layout(3, 512, 64) == kvr.E_ARG
    assert kvr.lib().kvr_row_layout(-1, 512, 64) == kvr.E_ARG


def test_null_contexts_and_calls():
    lib = kvr.lib()
    pack, attend = kvr.PackCall(), kvr.AttendCall()
    for name, args in (("kvr_pack_rows", (ctypes.byref(pack), None)),
                       ("kvr_attend_rows", (ctypes.byref(attend), None)),
                       ("kvr_bind_page_refs", (None,)), ("kvr_count_page_refs", (None,)),
                       ("kvr_release_requests", (0, None, None, None)),
                       ("kvr_fork_requests", (0, None, None, None, None)),
                       ("kvr_copy_pages", (0, None, None, None, None, None)),
                       ("kvr_pool_workspace", ()),
                       ("kvr_list_free_pages", (None, None, None, 0, None)),
                       ("kvr_compact_pool", (0, None, None, None, 0, None))):
        assert getattr(lib, name)(None, *args) == kvr.E_ARG, name
        assert "null context" in kvr.last_error()


def test_call_structs_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kvr.h")).read(),
                  flags=re.S)
    c_types = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float,
               "size_t": ctypes.c_size_t}
    for struct, cls in (("kvr_pack_call", kvr.PackCall), ("kvr_attend_call", kvr.AttendCall)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), text, re.S).group(1)
        want = []
        for line in filter(None, (x.strip() for x in body.split(";"))):
            name = re.search(r"(\w+)$", line).group(1)
            want.append((name, ctypes.c_void_p if "*" in line else c_types[line.split()[0]]))
        assert want == list(cls._fields_), struct


def test_row_formats_match_the_header():
    text = open(os.path.join(ROOT, "include", "kvr.h")).read()
    formats = {n.lower(): int(v) for n, v in re.findall(r"KVR_ROW_([A-Z0-9]+)\s*=\s*(\d+)", text)}
    assert formats == kvr.ROW_FORMATS
    values = {n: int(v) for n, v in re.findall(r"KVR_VALUE_([A-Z0-9]+)\s*=\s*(\d+)", text)}
    assert values == {"BF16": kvr._VALUE_TYPES["bfloat16"], "F16": kvr._VALUE_TYPES["float16"],
                      "F32": kvr._VALUE_TYPES["float32"]}


@pytest.mark.parametrize("args", [(-1, 1, 1, 512, 8), (1, 0, 1, 512, 8), (1, 1, 0, 512, 8),
                                  (1, 1, 1, 512, -1), (1, 1, 1, 384, 8), (1, 5000, 1, 512, 8),
                                  (1, 1, 5000, 512, 8), (1, 1, 1, 512, (1 << 24) + 1),
                                  (1 << 20, 4, 128, 512, 8)])
def test_attend_workspace_refuses(args):
    with pytest.raises(kvr.KvrError):
        kvr.Context.attend_workspace(*args)


def test_attend_workspace_covers_smaller_calls():
    """The workspace of a size serves every smaller one."""
    size = kvr.Context.attend_workspace
    most = size(64, 4, 128, 512, 2048)
    assert most >= 0
    for n in (0, 1, 2, 3, 7, 33, 64):
        for nq in (1, 3, 4):
            for heads in (1, 16, 17, 40, 64, 128):
                for rows in (0, 1, 64, 65, 700, 2048):
                    assert 0 <= size(n, nq, heads, 512, rows) <= most
                    assert size(n, nq, heads, 256, rows) <= size(n, nq, heads, 512, rows)


def test_binding_checks():
    with pytest.raises(TypeError, match="q: expected a GPU tensor, got <class 'int'>"):
        kvr._typed(5, "q", ("bfloat16",))
    with pytest.raises(TypeError, match="got one on cpu"):
        kvr._typed(torch.zeros(4), "latent", ("float32",))
    with pytest.raises(TypeError, match="expected a GPU tensor"):
        kvr._dev_here(torch.zeros(4), "loc", 16)
    with pytest.raises(TypeError, match="loc: expected int32 or uint32, got torch.int64"):
        kvr._words(torch.zeros(4, dtype=torch.int64), "loc", 4)
    with pytest.raises(TypeError, match="loc: expected a GPU tensor"):
        kvr._words(torch.zeros(4, dtype=torch.int32), "loc", 4)
    assert kvr._words(4096, "loc", 1 << 40) == 4096 and kvr._words(None, "loc", 4) is None
    assert kvr._dev_here(4096, "loc", 1 << 40) == 4096 and kvr._dev_here(None, "loc") is None
    assert kvr._workspace(None) == (None, 0)
    assert kvr._workspace(4096)[0] == 4096
    with pytest.raises(TypeError, match="workspace: expected a GPU tensor"):
        kvr._workspace(torch.zeros(4))
