"""Without a GPU: the drafter's K/V calls refuse a stream of another device than the
ring's.  A child process gives the library two small functions in place of the
runtime's: the current device is 0, and the stream at address 32 is device 1's."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

import pytest

from hierarchical_sparse_kv_resolve_amd import kvr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DEVICES = """
int hipGetDevice(int *device) { *device = 0; return 0; }
int hipStreamGetDevice(void *stream, int *device) { *device = stream == (void *)32; return 0; }
"""

CHILD = """
import ctypes, sys
ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
from hierarchical_sparse_kv_resolve_amd import kvr
L = kvr.lib()
h = ctypes.c_void_p()
assert L.kvr_draft_create(2, 64, 128, 0, None, 4096, 8192, ctypes.byref(h)) == 0, kvr.last_error()
assert L.kvr_draft_bind_kv(h, 1, 1, 64, 16, 16) == 0
write, attend = kvr.DraftWriteCall(), kvr.DraftAttendCall(nq=1, heads=1)
for stream, want in ((16, 0), (None, 0), (32, kvr.E_ARG)):  # calls of no entries launch nothing
    for call in (lambda: L.kvr_draft_write_kv(h, ctypes.byref(write), stream),
                 lambda: L.kvr_draft_read_kv(h, 0, 0, None, 0, None, None, None, None, stream),
                 lambda: L.kvr_draft_advance(h, 0, None, 1, None, None, stream),
                 lambda: L.kvr_draft_attend(h, ctypes.byref(attend), stream)):
        got = call()
        print(stream, got, kvr.last_error() if got else "")
        assert got == want
        assert not got or "the stream is on device 1, not the ring's device 0" in kvr.last_error()
"""


def test_streams_of_another_device(tmp_path):
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("gcc is not installed")
    kvr.lib()  # (built)
    src, lib = tmp_path / "devices.c", tmp_path / "libdevices.so"
    src.write_text(DEVICES)
    subprocess.run([gcc, "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    p = subprocess.run([sys.executable, "-c", CHILD, str(lib)], cwd=ROOT, capture_output=True,
                       text=True, timeout=120)
    assert p.returncode == 0, p.stdout[-2000:] + p.stderr[-2000:]
