"""Thin ctypes binding of libkvr.so (include/kvr.h).

Argument marshalling only: every entry point forwards raw device pointers,
sizes and a HIP stream to the C ABI, and raises KvrError on a non-OK return.
All work on the path runs in the library's HIP kernels; there is no fallback.
Tensors may be torch tensors (their data_ptr() is passed), plain integer
addresses, or None for NULL.  A torch tensor is checked against what the
header says of its argument (on the GPU or pinned host memory, contiguous, at
least the bytes the call reads or writes) before the call; addresses are
passed as given.  The stream defaults to torch's current stream.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvr.so")

OK = 0
E_ARG = -1
E_RANGE = -2
E_CAPACITY = -3
E_NO_HOST_COPY = -4
E_HIP = -5
E_STATE = -6

PLACE_TAIL, PLACE_PAGE, PLACE_HOT, PLACE_INVALID = 0, 1, 2, 3
LOC_INVALID = 0xFFFFFFFF
REUSE_SHARED_SOURCE = 0
REUSE_DISTINCT_PAYLOAD = 1

# Every entry point of include/kvr.h.
EXPORTS = ("kvr_create", "kvr_destroy", "kvr_last_error", "kvr_bind_metadata", "kvr_bind_layer",
           "kvr_init_state", "kvr_append_rows", "kvr_resolve_rows", "kvr_append_resolve_rows",
           "kvr_append_resolve_rows_deferred", "kvr_gather_rows", "kvr_fused_gather_append_rows",
           "kvr_gather_resolve_rows",
           "kvr_dedup_verify_selections", "kvr_reuse_locations", "kvr_status_summary",
           "kvr_host_alloc", "kvr_host_free", "kvr_timing_begin", "kvr_timing_end",
           "kvr_reclaim_pages", "kvr_restore_pages", "kvr_gather_resident_rows",
           "kvr_fill_gather_rows", "kvr_fused_gather_rows", "kvr_residency_create",
           "kvr_residency_destroy", "kvr_residency_admit", "kvr_residency_release",
           "kvr_residency_refill", "kvr_residency_counts", "kvr_draft_create",
           "kvr_draft_destroy", "kvr_draft_reset", "kvr_draft_append", "kvr_draft_rollback",
           "kvr_draft_window", "kvr_staging_create", "kvr_staging_destroy",
           "kvr_staging_acquire", "kvr_staging_release", "kvr_row_layout", "kvr_pack_rows",
           "kvr_attend_rows", "kvr_attend_workspace", "kvr_bind_page_refs", "kvr_count_page_refs",
           "kvr_release_requests", "kvr_fork_requests", "kvr_copy_pages", "kvr_pool_workspace",
           "kvr_list_free_pages", "kvr_compact_pool", "kvr_rotate_rows", "kvr_rope_frequencies",
           "kvr_token_logprobs", "kvr_logprob_workspace", "kvr_draft_bind_kv",
           "kvr_draft_write_kv", "kvr_draft_read_kv", "kvr_draft_advance", "kvr_draft_attend",
           "kvr_draft_attend_workspace")

# kvr_kernel: kinds of the library's kernel launches (launch timing).
KERNEL_NAMES = ("append", "resolve", "refill", "gather", "dedup", "state", "fused", "step",
                "attend", "pack", "pages", "rotate", "logprob")

# kvr_row_format, and the 16-bit type of queries, outputs and rope parts.
ROW_FORMATS = {"bf16": 0, "f16": 1, "fp8": 2}
_ROW_TYPES = {"bf16": "bfloat16", "f16": "float16", "fp8": "bfloat16"}
# kvr_value_type by torch dtype name.
_VALUE_TYPES = {"bfloat16": 0, "float16": 1, "float32": 2}
# kvr_rope_layout, kvr_rope_scaling, kvr_draft_mask.
ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp": 3}
DRAFT_MASKS = {"causal": 0, "block": 1, "kept": 2}
DRAFT_BLOCK = 64


class KvrError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"kvr error {code}: {msg}")
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [("n_req", ctypes.c_int32), ("n_layers", ctypes.c_int32),
                ("history_rows", ctypes.c_int32), ("max_new_rows", ctypes.c_int32),
                ("page_rows", ctypes.c_int32), ("tail_rows", ctypes.c_int32),
                ("hot_slots", ctypes.c_int32), ("row_bytes", ctypes.c_int32),
                ("sel_cap", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("pool_pages", ctypes.c_int64)]


STATS_FIELDS = ("calls", "tail", "page", "hit", "miss", "fill", "host_bytes", "error")


class GatherCall(ctypes.Structure):
    """kvr_gather_call of include/kvr.h."""
    _fields_ = [("n_layers", ctypes.c_int32), ("layers", ctypes.c_void_p),
                ("n", ctypes.c_int32), ("req_ids", ctypes.c_void_p), ("loc", ctypes.c_void_p),
                ("sel", ctypes.c_void_p), ("count", ctypes.c_void_p), ("stride", ctypes.c_int32),
                ("out", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("new_rows", ctypes.c_void_p), ("append_pos", ctypes.c_void_p)]


class ResolveCall(ctypes.Structure):
    """kvr_resolve_call of include/kvr.h."""
    _fields_ = [("n", ctypes.c_int32), ("req_ids", ctypes.c_void_p),
                ("new_rows", ctypes.c_void_p), ("append_status", ctypes.c_void_p),
                ("append_pos", ctypes.c_void_p), ("sel", ctypes.c_void_p),
                ("sel_count", ctypes.c_void_p), ("stride", ctypes.c_int32),
                ("loc", ctypes.c_void_p), ("fills", ctypes.c_void_p),
                ("fill_count", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("stats", ctypes.c_void_p)]


class PackCall(ctypes.Structure):
    """kvr_pack_call of include/kvr.h."""
    _fields_ = [("format", ctypes.c_int32), ("value_type", ctypes.c_int32), ("n", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("d_rope", ctypes.c_int32), ("eps", ctypes.c_float),
                ("latent", ctypes.c_void_p), ("rope", ctypes.c_void_p),
                ("weight", ctypes.c_void_p), ("rows", ctypes.c_void_p),
                ("latent_stride", ctypes.c_int64), ("rope_stride", ctypes.c_int64)]


class AttendCall(ctypes.Structure):
    """kvr_attend_call of include/kvr.h."""
    _fields_ = [("layer", ctypes.c_int32), ("format", ctypes.c_int32), ("n", ctypes.c_int32),
                ("nq", ctypes.c_int32), ("heads", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("d_rope", ctypes.c_int32), ("stride", ctypes.c_int32), ("k", ctypes.c_int32),
                ("scale", ctypes.c_float), ("req_ids", ctypes.c_void_p), ("loc", ctypes.c_void_p),
                ("rows", ctypes.c_void_p), ("count", ctypes.c_void_p), ("map", ctypes.c_void_p),
                ("q", ctypes.c_void_p), ("q_stride_entry", ctypes.c_int64),
                ("q_stride_query", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class RotatePart(ctypes.Structure):
    """kvr_rotate_part of include/kvr.h."""
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("x_stride_token", ctypes.c_int64), ("x_stride_head", ctypes.c_int64),
                ("out_stride_token", ctypes.c_int64), ("out_stride_head", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("d_head", ctypes.c_int32), ("at", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class RotateCall(ctypes.Structure):
    """kvr_rotate_call of include/kvr.h."""
    _fields_ = [("value_type", ctypes.c_int32), ("layout", ctypes.c_int32), ("n", ctypes.c_int32),
                ("d_rot", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("inverse", ctypes.c_int32), ("positions", ctypes.c_void_p),
                ("frequencies", ctypes.c_void_p), ("query", RotatePart), ("key", RotatePart)]


class LogprobCall(ctypes.Structure):
    """kvr_logprob_call of include/kvr.h."""
    _fields_ = [("value_type", ctypes.c_int32), ("n", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("m", ctypes.c_int32), ("top", ctypes.c_int32), ("scale", ctypes.c_float),
                ("logits", ctypes.c_void_p), ("logits_stride", ctypes.c_int64),
                ("tokens", ctypes.c_void_p), ("logprob", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("entropy", ctypes.c_void_p),
                ("top_ids", ctypes.c_void_p), ("top_logprob", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class DraftWriteCall(ctypes.Structure):
    """kvr_draft_write_call of include/kvr.h."""
    _fields_ = [("layer", ctypes.c_int32), ("value_type", ctypes.c_int32), ("n", ctypes.c_int32),
                ("rows", ctypes.c_int32), ("req_ids", ctypes.c_void_p),
                ("count", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_stride_entry", ctypes.c_int64), ("k_stride_token", ctypes.c_int64),
                ("k_stride_head", ctypes.c_int64), ("v_stride_entry", ctypes.c_int64),
                ("v_stride_token", ctypes.c_int64), ("v_stride_head", ctypes.c_int64),
                ("status", ctypes.c_void_p)]


class DraftAttendCall(ctypes.Structure):
    """kvr_draft_attend_call of include/kvr.h."""
    _fields_ = [("layer", ctypes.c_int32), ("mask", ctypes.c_int32), ("n", ctypes.c_int32),
                ("nq", ctypes.c_int32), ("heads", ctypes.c_int32), ("scale", ctypes.c_float),
                ("req_ids", ctypes.c_void_p), ("count", ctypes.c_void_p), ("q", ctypes.c_void_p),
                ("q_stride_entry", ctypes.c_int64), ("q_stride_query", ctypes.c_int64),
                ("q_stride_head", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


_lib = None


def lib():
    """Load libkvr.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m hierarchical_sparse_kv_resolve_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, U = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        sig = {
            "kvr_create": [P, P],
            "kvr_destroy": [P],
            "kvr_bind_metadata": [P, P, P, P, P, P, P],
            "kvr_bind_layer": [P, I, P, P, P, P],
            "kvr_init_state": [P, P],
            "kvr_append_rows": [P, I, P, P, P, P],
            "kvr_resolve_rows": [P, I, P, P, P, I, P, P, P, I, P, P, P],
            "kvr_append_resolve_rows": [P, I, P, P, P, P, P, I, P, P, P, I, P, P, P],
            "kvr_append_resolve_rows_deferred": [P, I, P, P, P, P, P, P, I, P, P, P, I, P, P, P],
            "kvr_gather_rows": [P, I, P, I, P, P, P, I, P, P, P],
            "kvr_gather_resident_rows": [P, I, P, I, P, P, P, I, P, P, P],
            "kvr_fill_gather_rows": [P, I, P, I, P, P, P, P, I, P, P, P],
            "kvr_fused_gather_rows": [P, I, P, I, P, P, P, P, I, P, P, P],
            "kvr_fused_gather_append_rows": [P, I, P, I, P, P, P, P, I, P, P, P, P, P],
            "kvr_gather_resolve_rows": [P, P, P, P],
            "kvr_dedup_verify_selections": [P, I, I, I, P, P, P, P, P],
            "kvr_reuse_locations": [P, I, I, P, I, P, P, P, P, I, P, P, P, P],
            "kvr_status_summary": [P, I, P],
            "kvr_host_alloc": [U, P],
            "kvr_host_free": [P],
            "kvr_timing_begin": [P, I],
            "kvr_timing_end": [P, I, P, P, P],
            "kvr_reclaim_pages": [P, I, P, P, P, P, P],
            "kvr_restore_pages": [P, I, P, P, P, P, P],
            "kvr_residency_create": [I, I, I, ctypes.c_int64, P, P],
            "kvr_residency_destroy": [P],
            "kvr_residency_admit": [P, ctypes.c_int64, I, P, I, P, P, P, P],
            "kvr_residency_release": [P, I],
            "kvr_residency_refill": [P, I, I, P, P, P, P],
            "kvr_residency_counts": [P, P, P, P],
            "kvr_draft_create": [I, I, I, I, P, P, P, P],
            "kvr_draft_destroy": [P],
            "kvr_draft_reset": [P, P],
            "kvr_draft_append": [P, I, P, I, P, P, P],
            "kvr_draft_rollback": [P, I, P, P, P, P],
            "kvr_draft_window": [P, I, P, P, P, P, P],
            "kvr_staging_create": [I, P],
            "kvr_staging_destroy": [P],
            "kvr_staging_acquire": [P, P, P],
            "kvr_staging_release": [P, I, P],
            "kvr_row_layout": [I, I, I],
            "kvr_pack_rows": [P, P, P],
            "kvr_attend_rows": [P, P, P],
            "kvr_attend_workspace": [I, I, I, I, I],
            "kvr_bind_page_refs": [P, P],
            "kvr_count_page_refs": [P, P],
            "kvr_release_requests": [P, I, P, P, P],
            "kvr_fork_requests": [P, I, P, P, P, P],
            "kvr_copy_pages": [P, I, P, P, P, P, P],
            "kvr_pool_workspace": [P],
            "kvr_list_free_pages": [P, P, P, P, U, P],
            "kvr_compact_pool": [P, I, P, P, P, U, P],
            "kvr_rotate_rows": [P, P, P],
            "kvr_rope_frequencies": [I, ctypes.c_double, I, ctypes.c_double, I, ctypes.c_double,
                                     ctypes.c_double, P, P],
            "kvr_token_logprobs": [P, P, P],
            "kvr_logprob_workspace": [I, I],
            "kvr_draft_bind_kv": [P, I, I, I, P, P],
            "kvr_draft_write_kv": [P, P, P],
            "kvr_draft_read_kv": [P, I, I, P, I, P, P, P, P, P],
            "kvr_draft_advance": [P, I, P, I, P, P, P],
            "kvr_draft_attend": [P, P, P],
            "kvr_draft_attend_workspace": [P, I, I, I],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        for name in ("kvr_attend_workspace", "kvr_pool_workspace", "kvr_logprob_workspace",
                     "kvr_draft_attend_workspace"):
            getattr(L, name).restype = ctypes.c_int64
        L.kvr_last_error.argtypes = []
        L.kvr_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if hasattr(x, "ctypes"):  # numpy array (host memory)
        return x.ctypes.data
    raise TypeError(f"cannot take the address of {type(x)}")


def _dev(x, name: str, nbytes: int = 0) -> int | None:
    """Address of a device argument.  A torch tensor must live on the GPU, be
    contiguous and hold at least `nbytes` (the size the header's layout gives
    it for this call), so that a host tensor or a short buffer raises here
    instead of reaching a kernel.  Integer addresses and None pass unchecked."""
    if x is None or isinstance(x, int):
        return x
    if hasattr(x, "is_cuda"):
        if not x.is_cuda:
            raise TypeError(f"{name}: expected a GPU tensor, got one on {x.device}")
        if not x.is_contiguous():
            raise ValueError(f"{name}: the tensor is not contiguous")
        have = x.numel() * x.element_size()
        if have < nbytes:
            raise ValueError(f"{name}: {have} bytes, the call needs {nbytes}")
        return x.data_ptr()
    raise TypeError(f"{name}: expected a GPU tensor or an address, got {type(x)}")


def _pinned(x, name: str, nbytes: int = 0) -> int | None:
    """Address of a pinned host argument (a torch tensor in pinned CPU memory,
    or an address from host_alloc)."""
    if x is None or isinstance(x, int):
        return x
    if hasattr(x, "is_cuda"):
        if x.is_cuda or not x.is_pinned():
            raise TypeError(f"{name}: expected a pinned host tensor")
        if not x.is_contiguous():
            raise ValueError(f"{name}: the tensor is not contiguous")
        have = x.numel() * x.element_size()
        if have < nbytes:
            raise ValueError(f"{name}: {have} bytes, the call needs {nbytes}")
        return x.data_ptr()
    raise TypeError(f"{name}: expected a pinned host tensor or an address, got {type(x)}")


def _stream(stream, here: int | None = None) -> int | None:
    if stream is None:
        if _raw_stream is not None and here is not None:
            return _raw_stream(here)
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:  # without building a Stream object for each call
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int):
    if rc != OK:
        raise KvrError(rc, lib().kvr_last_error().decode())
    return rc


_get_device = _raw_stream = None  # torch's, once it has initialised the GPU


def _here() -> int:
    """The current device (which the library requires to be the context's)."""
    global _get_device, _raw_stream
    if _get_device is None:
        import torch
        here = torch.cuda.current_device()
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        return here
    return _get_device()


def _typed(x, name: str, dtypes, here: int | None = None, shape=None):
    """A strided tensor on the current device (`here`), of one of the dtypes
    (names), whose last dimension is contiguous; its dtype's name."""
    try:  # (all as it should be, in few steps; else what is wrong is found below)
        kind = _DTYPE_NAMES[x.dtype]
        if (kind in dtypes and x.get_device() == here and (shape is None or x.shape == shape)
                and (x.is_contiguous() or x.stride(-1) == 1)):
            return kind
    except (AttributeError, KeyError, IndexError, RuntimeError):
        pass
    if not getattr(x, "is_cuda", False):
        what = f"one on {x.device}" if hasattr(x, "is_cuda") else type(x)
        raise TypeError(f"{name}: expected a GPU tensor, got {what}")
    kind = _DTYPE_NAMES.get(x.dtype)
    if kind is None:
        kind = _DTYPE_NAMES[x.dtype] = str(x.dtype)[6:]
    if kind not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(dtypes)}, got {x.dtype}")
    if shape is not None and x.shape != shape:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, the call needs {tuple(shape)}")
    if not x.is_contiguous() and x.numel() and x.shape[-1] > 1 and x.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension is not contiguous")
    _same_device(x, name, here)
    return kind


_DTYPE_NAMES: dict = {}
_NO_PART = (None, None, 0, 0, 0, 0, 0, 0, 0, 0)


def _same_device(x, name: str, here: int | None = None):
    """A tensor of another device than the current one is refused; addresses
    pass."""
    if getattr(x, "is_cuda", False):
        here = _here() if here is None else here
        if x.get_device() != here:
            raise ValueError(f"{name}: on {x.device}, the current device is cuda:{here}")
    return x


def _full(x, name: str, kind: str, here: int, shape) -> int:
    """Address of a contiguous tensor of one dtype (by name) and shape on the
    current device."""
    if _typed(x, name, (kind,), here, shape) and x.is_contiguous():
        return x.data_ptr()
    return _dev(x, name)


def _dev_here(x, name: str, nbytes: int = 0, here: int | None = None) -> int | None:
    if x is None or isinstance(x, int):
        return x
    return _dev(_same_device(x, name, here), name, nbytes)


def _words(x, name: str, n: int, here: int | None = None) -> int | None:
    """Address of n 32-bit integers on the current device."""
    if x is None or isinstance(x, int):
        return x
    try:
        if (_DTYPE_NAMES[x.dtype] in ("int32", "uint32") and x.get_device() == here
                and x.is_contiguous() and x.numel() >= n):
            return x.data_ptr()
    except (AttributeError, KeyError, RuntimeError):
        pass
    if hasattr(x, "is_cuda"):
        kind = _DTYPE_NAMES.get(x.dtype)
        if kind is None:
            kind = _DTYPE_NAMES[x.dtype] = str(x.dtype)[6:]
        if kind != "int32" and kind != "uint32":
            raise TypeError(f"{name}: expected int32 or uint32, got {x.dtype}")
    return _dev_here(x, name, 4 * n, here)


def _workspace(x, here: int | None = None):
    """(address, bytes) of a workspace tensor; an address is taken to hold what
    the call needs."""
    if x is None or isinstance(x, int):
        return x, (1 << 62 if x else 0)
    return _dev_here(x, "workspace", 0, here), x.numel() * x.element_size()


def row_layout(fmt: str, d_v: int, d_rope: int) -> int:
    """Bytes of one row of a format ("bf16", "f16" or "fp8")."""
    rc = lib().kvr_row_layout(_row_format(fmt), d_v, d_rope)
    return rc if rc >= 0 else _check(rc)


def _row_format(fmt: str) -> int:
    if fmt not in ROW_FORMATS:
        raise ValueError(f"unknown row format {fmt!r}: one of {', '.join(ROW_FORMATS)}")
    return ROW_FORMATS[fmt]


def _choice(value: str, what: str, of: dict) -> int:
    if value not in of:
        raise ValueError(f"unknown {what} {value!r}: one of {', '.join(of)}")
    return of[value]


def rope_frequencies(d_rot, base=10000.0, scaling="none", factor=1.0, original_length=0,
                     beta_fast=32.0, beta_slow=1.0):
    """(float64 array [d_rot / 2] of turns per position, magnitude): what
    Context.rotate_rows takes.  scaling: "none", "linear", "base" or "ramp"; see
    kvr_rope_scaling."""
    import numpy as np
    kind = _choice(scaling, "scaling", ROPE_SCALINGS)
    out = np.zeros(max(1, d_rot // 2), dtype=np.float64)
    magnitude = ctypes.c_float()
    _check(lib().kvr_rope_frequencies(d_rot, base, kind, factor, original_length, beta_fast,
                                      beta_slow, out.ctypes.data, ctypes.byref(magnitude)))
    return out, magnitude.value


def last_error() -> str:
    return lib().kvr_last_error().decode()


def host_alloc(nbytes: int) -> int:
    out = ctypes.c_void_p()
    _check(lib().kvr_host_alloc(nbytes, ctypes.byref(out)))
    return out.value


def host_free(ptr: int) -> None:
    _check(lib().kvr_host_free(ptr))


def status_summary(status_host) -> tuple[int, int]:
    """(number of failed requests, index of the first or -1) of a host int32 array."""
    import numpy as np
    st = np.ascontiguousarray(status_host, dtype=np.int32)
    first = ctypes.c_int32()
    bad = lib().kvr_status_summary(st.ctypes.data, len(st), ctypes.byref(first))
    if bad < 0:
        _check(bad)
    return bad, first.value


class Context:
    """One KV source: n_req requests and n_layers payload layers."""

    def __init__(self, *, n_req, n_layers, history_rows, max_new_rows, page_rows, tail_rows,
                 hot_slots, row_bytes, sel_cap, pool_pages):
        self.cfg = Config(n_req, n_layers, history_rows, max_new_rows, page_rows, tail_rows,
                          hot_slots, row_bytes, sel_cap, 0, pool_pages)
        h = ctypes.c_void_p()
        _check(lib().kvr_create(ctypes.byref(self.cfg), ctypes.byref(h)))
        self.handle = h.value
        self._keep = []

    def close(self):
        if self.handle:
            lib().kvr_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _sizes(self):
        c = self.cfg
        return (c.n_req, c.n_layers, c.history_rows, c.max_new_rows, c.page_rows, c.tail_rows,
                c.hot_slots, c.row_bytes, c.pool_pages)

    def bind_metadata(self, L, page_map, host_valid, tag, stamp, clock):
        N, _, H, _, P, _, B, _, _ = self._sizes()
        npg = (H + P - 1) // P if P > 0 else 0
        _check(lib().kvr_bind_metadata(self.handle, _dev(L, "L", 4 * N),
                                       _dev(page_map, "page_map", 4 * N * npg),
                                       _dev(host_valid, "host_valid", N * npg),
                                       _dev(tag, "tag", 4 * N * B), _dev(stamp, "stamp", 4 * N * B),
                                       _dev(clock, "clock", 4 * N)))

    def bind_layer(self, layer, tail, pool, hot, host):
        N, _, H, M, P, T, B, R, pool_pages = self._sizes()
        _check(lib().kvr_bind_layer(self.handle, layer, _dev(tail, "tail", N * T * R),
                                    _dev(pool, "pool", pool_pages * P * R),
                                    _dev(hot, "hot", N * B * R),
                                    _pinned(host, "host", N * (H + M) * R)))

    def init_state(self, stream=None):
        _check(lib().kvr_init_state(self.handle, _stream(stream)))

    def append_rows(self, n, req_ids, new_rows, status=None, stream=None):
        _, NL, _, _, _, _, _, R, _ = self._sizes()
        _check(lib().kvr_append_rows(self.handle, n, _dev(req_ids, "req_ids", 4 * n),
                                     _dev(new_rows, "new_rows", NL * n * R),
                                     _dev(status, "status", 4 * n), _stream(stream)))

    def _resolve_args(self, n, req_ids, sel, sel_count, stride, loc, fills, fill_count, status,
                      stats):
        B = self.cfg.hot_slots
        m = max(n, 0) * max(stride, 0)
        return (_dev(req_ids, "req_ids", 4 * n), _dev(sel, "sel", 4 * m),
                _dev(sel_count, "sel_count", 4 * n), _dev(loc, "loc", 4 * m),
                _dev(fills, "fills", 8 * n * B), _dev(fill_count, "fill_count", 4 * n),
                _dev(status, "status", 4 * n), _dev(stats, "stats", 8 * len(STATS_FIELDS)))

    def resolve_rows(self, n, req_ids, sel, sel_count, stride, loc, fills, fill_count, fill_layer,
                     status, stats=None, stream=None):
        rid, sl, sc, lc, fl, fc, st, sts = self._resolve_args(n, req_ids, sel, sel_count, stride,
                                                              loc, fills, fill_count, status,
                                                              stats)
        _check(lib().kvr_resolve_rows(self.handle, n, rid, sl, sc, stride, lc, fl, fc, fill_layer,
                                      st, sts, _stream(stream)))

    def append_resolve_rows(self, n, req_ids, new_rows, append_status, sel, sel_count, stride, loc,
                            fills, fill_count, fill_layer, status, stats=None, stream=None):
        NL, R = self.cfg.n_layers, self.cfg.row_bytes
        rid, sl, sc, lc, fl, fc, st, sts = self._resolve_args(n, req_ids, sel, sel_count, stride,
                                                              loc, fills, fill_count, status,
                                                              stats)
        _check(lib().kvr_append_resolve_rows(self.handle, n, rid,
                                             _dev(new_rows, "new_rows", NL * n * R),
                                             _dev(append_status, "append_status", 4 * n), sl, sc,
                                             stride, lc, fl, fc, fill_layer, st, sts,
                                             _stream(stream)))

    def append_resolve_rows_deferred(self, n, req_ids, new_rows, append_status, append_pos, sel,
                                     sel_count, stride, loc, fills, fill_count, fill_layer,
                                     status, stats=None, stream=None):
        NL, R = self.cfg.n_layers, self.cfg.row_bytes
        rid, sl, sc, lc, fl, fc, st, sts = self._resolve_args(n, req_ids, sel, sel_count, stride,
                                                              loc, fills, fill_count, status,
                                                              stats)
        _check(lib().kvr_append_resolve_rows_deferred(
            self.handle, n, rid, _dev(new_rows, "new_rows", NL * n * R),
            _dev(append_status, "append_status", 4 * n), _dev(append_pos, "append_pos", 4 * n),
            sl, sc, stride, lc, fl, fc, fill_layer, st, sts, _stream(stream)))

    def _gather_args(self, layers, n, req_ids, loc, count, stride, outs, status):
        nl = len(layers)
        m = max(n, 0) * max(stride, 0)
        R = self.cfg.row_bytes
        if len(outs) != nl:
            raise ValueError(f"outs: {len(outs)} buffers for {nl} layers")
        arr_l = (ctypes.c_int32 * max(1, nl))(*layers)
        arr_o = (ctypes.c_void_p * max(1, nl))(*[_dev(o, "out", m * R) for o in outs])
        return (nl, arr_l, _dev(req_ids, "req_ids", 4 * n), _dev(loc, "loc", 4 * m),
                _dev(count, "count", 4 * n), arr_o, _dev(status, "status", 4 * n))

    def gather_rows(self, layers, n, req_ids, loc, count, stride, outs, status=None, stream=None):
        nl, arr_l, rid, lc, cnt, arr_o, st = self._gather_args(layers, n, req_ids, loc, count,
                                                               stride, outs, status)
        _check(lib().kvr_gather_rows(self.handle, nl, arr_l, n, rid, lc, cnt, stride, arr_o, st,
                                     _stream(stream)))

    def gather_resident_rows(self, layers, n, req_ids, loc, count, stride, outs, status=None,
                             stream=None):
        nl, arr_l, rid, lc, cnt, arr_o, st = self._gather_args(layers, n, req_ids, loc, count,
                                                               stride, outs, status)
        _check(lib().kvr_gather_resident_rows(self.handle, nl, arr_l, n, rid, lc, cnt, stride,
                                              arr_o, st, _stream(stream)))

    def fill_gather_rows(self, layers, n, req_ids, loc, sel, count, stride, outs, status=None,
                         stream=None):
        nl, arr_l, rid, lc, cnt, arr_o, st = self._gather_args(layers, n, req_ids, loc, count,
                                                               stride, outs, status)
        sl = _dev(sel, "sel", 4 * max(n, 0) * max(stride, 0))
        _check(lib().kvr_fill_gather_rows(self.handle, nl, arr_l, n, rid, lc, sl, cnt, stride,
                                          arr_o, st, _stream(stream)))

    def fused_gather_rows(self, layers, n, req_ids, loc, sel, count, stride, outs, status=None,
                          stream=None):
        nl, arr_l, rid, lc, cnt, arr_o, st = self._gather_args(layers, n, req_ids, loc, count,
                                                               stride, outs, status)
        sl = _dev(sel, "sel", 4 * max(n, 0) * max(stride, 0))
        _check(lib().kvr_fused_gather_rows(self.handle, nl, arr_l, n, rid, lc, sl, cnt, stride,
                                           arr_o, st, _stream(stream)))

    def fused_gather_append_rows(self, layers, n, req_ids, loc, sel, count, stride, outs,
                                 new_rows, append_pos, status=None, stream=None):
        nl, arr_l, rid, lc, cnt, arr_o, st = self._gather_args(layers, n, req_ids, loc, count,
                                                               stride, outs, status)
        sl = _dev(sel, "sel", 4 * max(n, 0) * max(stride, 0))
        NL, R = self.cfg.n_layers, self.cfg.row_bytes
        _check(lib().kvr_fused_gather_append_rows(
            self.handle, nl, arr_l, n, rid, lc, sl, cnt, stride, arr_o, st,
            _dev(new_rows, "new_rows", NL * n * R), _dev(append_pos, "append_pos", 4 * n),
            _stream(stream)))

    def gather_resolve_rows(self, gather=None, resolve=None, stream=None):
        """kvr_gather_resolve_rows.  gather: dict(layers, n, req_ids, loc, sel,
        count, stride, outs, status, new_rows, append_pos) or None; resolve:
        dict(n, req_ids, new_rows, append_status, append_pos, sel, sel_count,
        stride, loc, fills, fill_count, status, stats) or None.  Missing keys
        are NULL."""
        keep = []
        g_ptr = r_ptr = None
        NL, R = self.cfg.n_layers, self.cfg.row_bytes
        if gather is not None:
            g = {**dict(req_ids=None, count=None, status=None, new_rows=None, append_pos=None,
                        sel=None), **gather}
            n, stride = g["n"], g["stride"]
            nl, arr_l, rid, lc, cnt, arr_o, st = self._gather_args(
                g["layers"], n, g["req_ids"], g["loc"], g["count"], stride, g["outs"], g["status"])
            gc = GatherCall(nl, ctypes.addressof(arr_l), n, rid, lc,
                            _dev(g["sel"], "sel", 4 * max(n, 0) * max(stride, 0)), cnt, stride,
                            ctypes.addressof(arr_o), st,
                            _dev(g["new_rows"], "new_rows", NL * n * R),
                            _dev(g["append_pos"], "append_pos", 4 * n))
            keep += [arr_l, arr_o, gc]
            g_ptr = ctypes.addressof(gc)
        if resolve is not None:
            r = {**dict(req_ids=None, new_rows=None, append_status=None, append_pos=None,
                        sel_count=None, stats=None), **resolve}
            n = r["n"]
            rid, sl, sc, lc, fl, fc, st, sts = self._resolve_args(
                n, r["req_ids"], r["sel"], r["sel_count"], r["stride"], r["loc"], r["fills"],
                r["fill_count"], r["status"], r["stats"])
            rc = ResolveCall(n, rid, _dev(r["new_rows"], "new_rows", NL * n * R),
                             _dev(r["append_status"], "append_status", 4 * n),
                             _dev(r["append_pos"], "append_pos", 4 * n), sl, sc, r["stride"], lc,
                             fl, fc, st, sts)
            keep.append(rc)
            r_ptr = ctypes.addressof(rc)
        _check(lib().kvr_gather_resolve_rows(self.handle, g_ptr, r_ptr, _stream(stream)))

    def dedup_verify_selections(self, n, q, k, sel, union_rows, union_count, map_, stream=None):
        m = max(n, 0) * max(q, 0) * max(k, 0)
        _check(lib().kvr_dedup_verify_selections(self.handle, n, q, k, _dev(sel, "sel", 4 * m),
                                                 _dev(union_rows, "union_rows", 4 * m),
                                                 _dev(union_count, "union_count", 4 * n),
                                                 _dev(map_, "map", 4 * m), _stream(stream)))

    def timing_begin(self, capacity: int):
        """Record the duration of each kernel this context launches from now on
        (events on the launches themselves; measurement aid)."""
        _check(lib().kvr_timing_begin(self.handle, capacity))
        self._timing_cap = capacity

    def timing_end(self):
        """Stop recording; waits for the recorded launches.  Returns a list of
        (kernel name, milliseconds) in launch order."""
        import numpy as np
        cap = getattr(self, "_timing_cap", 0)
        kinds = np.zeros(max(1, cap), dtype=np.int32)
        ms = np.zeros(max(1, cap), dtype=np.float32)
        n = ctypes.c_int32()
        _check(lib().kvr_timing_end(self.handle, cap, kinds.ctypes.data, ms.ctypes.data,
                                    ctypes.byref(n)))
        m = min(n.value, cap)
        return [(KERNEL_NAMES[k], float(t)) for k, t in zip(kinds[:m], ms[:m])]

    def reclaim_pages(self, n, req_ids, pages, freed_phys, status=None, stream=None):
        _check(lib().kvr_reclaim_pages(self.handle, n, _dev(req_ids, "req_ids", 4 * n),
                                       _dev(pages, "pages", 4 * n),
                                       _dev(freed_phys, "freed_phys", 4 * n),
                                       _dev(status, "status", 4 * n), _stream(stream)))

    def restore_pages(self, n, req_ids, pages, phys, status=None, stream=None):
        _check(lib().kvr_restore_pages(self.handle, n, _dev(req_ids, "req_ids", 4 * n),
                                       _dev(pages, "pages", 4 * n), _dev(phys, "phys", 4 * n),
                                       _dev(status, "status", 4 * n), _stream(stream)))

    def reuse_locations(self, mode, dst_layers, n, req_ids, src_loc, dst_loc, count, stride,
                        fills=None, fill_count=None, status=None, stream=None):
        layers = list(dst_layers or [])
        arr_l = (ctypes.c_int32 * max(1, len(layers)))(*layers)
        m = max(n, 0) * max(stride, 0)
        B = self.cfg.hot_slots
        _check(lib().kvr_reuse_locations(self.handle, mode, len(layers), arr_l, n,
                                         _dev(req_ids, "req_ids", 4 * n),
                                         _dev(src_loc, "src_loc", 4 * m),
                                         _dev(dst_loc, "dst_loc", 4 * m),
                                         _dev(count, "count", 4 * n),
                                         stride, _dev(fills, "fills", 8 * n * B),
                                         _dev(fill_count, "fill_count", 4 * n),
                                         _dev(status, "status", 4 * n), _stream(stream)))

    # ------------------------------------------- rows in a model's format

    def pack_rows(self, n, latent, rope, rows, *, fmt, d_v, d_rope, weight=None, eps=0.0,
                  stream=None):
        """Rows of n tokens: latent [n, d_v] and rope [n, d_rope] (bf16, fp16 or
        fp32, both of one type; rows may be strided slices), normalised where a
        float32 weight [d_v] is given, into rows (n * row_bytes bytes, on the
        device or pinned)."""
        here = _here()
        kind = _typed(latent, "latent", _VALUE_TYPES, here, (n, d_v))
        if d_rope:
            _typed(rope, "rope", (kind,), here, (n, d_rope))
        if weight is not None:
            _typed(weight, "weight", ("float32",), here, (d_v,))
        need = max(n, 0) * self.cfg.row_bytes
        on_host = hasattr(rows, "is_cuda") and not rows.is_cuda
        call = PackCall(_row_format(fmt), _VALUE_TYPES[kind], n, d_v, d_rope, eps,
                        latent.data_ptr(), rope.data_ptr() if d_rope else None,
                        None if weight is None else weight.data_ptr(),
                        _pinned(rows, "rows", need) if on_host else
                        _dev_here(rows, "rows", need, here),
                        latent.stride(0), rope.stride(0) if d_rope else 0)
        _check(lib().kvr_pack_rows(self.handle, ctypes.byref(call), _stream(stream)))

    @staticmethod
    def attend_workspace(n, nq, heads, d_v, rows) -> int:
        """Workspace bytes for attend_rows calls of up to these sizes; rows is
        the rows per query (the map's k, or stride without a map)."""
        got = lib().kvr_attend_workspace(n, nq, heads, d_v, rows)
        return got if got >= 0 else _check(got)

    def attend_rows(self, layer, n, req_ids, q, out, *, fmt, d_v, d_rope, scale, stride, loc=None,
                    rows=None, count=None, map_=None, lse=None, status=None, workspace=None,
                    stream=None):
        """Attention of q [n, nq, heads, d_v + d_rope] over the rows that loc
        names in `layer` (or over the gathered rows), into out [n, nq, heads,
        d_v] and lse [n, nq, heads]; with map_ [n, nq, k] query a of entry i
        attends to the entries map_[i, a] only.  See kvr_attend_rows."""
        code, kind, here = _row_format(fmt), (_ROW_TYPES[fmt],), _here()
        if getattr(q, "ndim", 4) != 4:
            raise ValueError(f"q: {q.ndim} dimensions, the call needs [n, nq, heads, d_v + d_rope]")
        nq, heads = (int(q.shape[1]), int(q.shape[2])) if hasattr(q, "shape") else (1, 1)
        _typed(q, "q", kind, here, (n, nq, heads, d_v + d_rope))
        _typed(out, "out", kind, here, (n, nq, heads, d_v))
        if lse is not None:
            _typed(lse, "lse", ("float32",), here, (n, nq, heads))
        k = 0
        if map_ is not None:
            if getattr(map_, "ndim", 3) != 3:
                raise ValueError(f"map: {map_.ndim} dimensions, the call needs [n, nq, k]")
            k = int(map_.shape[2]) if hasattr(map_, "shape") else 0
            _typed(map_, "map", ("int32",), here, (n, nq, k))
        m = max(n, 0) * max(stride, 0)
        ws, ws_bytes = _workspace(workspace, here)
        strides = q.stride()
        call = AttendCall(layer, code, n, nq, heads, d_v, d_rope, stride, k, scale,
                          _words(req_ids, "req_ids", n, here),
                          _words(loc, "loc", m, here),
                          _dev_here(rows, "rows", m * self.cfg.row_bytes, here),
                          _words(count, "count", n, here), _dev(map_, "map"),
                          q.data_ptr(), strides[0], strides[1], strides[2], _dev(out, "out"),
                          _dev(lse, "lse"), _words(status, "status", n, here), ws, ws_bytes)
        _check(lib().kvr_attend_rows(self.handle, ctypes.byref(call), _stream(stream)))

    # ------------------------------------------- positions and scores

    def rotate_rows(self, n, positions, frequencies, x, out=None, key=None, key_out=None, *, d_rot,
                    layout, at=0, key_at=0, magnitude=1.0, inverse=False, stream=None):
        """Rotates values [at, at + d_rot) of each head of x [n, heads, d_head] by
        its token's position (int32 [n]) times the frequencies (float64
        [d_rot / 2], turns per position), into out (in place without it), and
        with them those of key [n, key heads, key d_head].  Last dimensions
        contiguous; x and key of one type, bf16, fp16 or fp32.  See
        kvr_rotate_rows."""
        here = _here()
        if x is None:
            if out is not None:
                raise ValueError("x: an output without an input")
            if key is None:
                raise ValueError("x or key is required")
            kind, first = None, _NO_PART
        else:
            kind, first = self._rotate_part(n, x, out, at, "x", _VALUE_TYPES, here)
        if key is None:
            if key_out is not None:
                raise ValueError("key: an output without an input")
            second = _NO_PART
        else:
            kind, second = self._rotate_part(n, key, key_out, key_at, "key",
                                             _VALUE_TYPES if kind is None else (kind,), here)
        freq = _full(frequencies, "frequencies", "float64", here, (d_rot // 2,))
        call = RotateCall(_VALUE_TYPES[kind], _choice(layout, "layout", ROPE_LAYOUTS), n, d_rot,
                          magnitude, inverse, _words(positions, "positions", n, here), freq, first,
                          second)
        _check(lib().kvr_rotate_rows(self.handle, ctypes.byref(call), _stream(stream, here)))

    @staticmethod
    def _rotate_part(n, src, dst, at, name, kinds, here):
        if getattr(src, "ndim", 3) != 3:
            raise ValueError(f"{name}: {src.ndim} dimensions, the call needs [n, heads, d_head]")
        kind = _typed(src, name, kinds, here)
        shape, a = src.shape, src.stride()
        if shape[0] != n:
            raise ValueError(f"{name}: {shape[0]} tokens, the call has {n}")
        if dst is None:
            p = src.data_ptr()
            return kind, (p, p, a[0], a[1], a[0], a[1], shape[1], shape[2], at, 0)
        _typed(dst, f"{name}'s output", (kind,), here, shape)
        b = dst.stride()
        return kind, (src.data_ptr(), dst.data_ptr(), a[0], a[1], b[0], b[1], shape[1], shape[2],
                      at, 0)

    @staticmethod
    def logprob_workspace(n, vocab) -> int:
        """Workspace bytes for token_logprobs calls of up to these sizes."""
        got = lib().kvr_logprob_workspace(n, vocab)
        return got if got >= 0 else _check(got)

    def token_logprobs(self, n, logits, tokens=None, logprob=None, *, lse=None, entropy=None,
                       top_ids=None, top_logprob=None, scale=1.0, workspace=None, stream=None):
        """Log probabilities [n, m] of tokens (int32 [n, m]) under rows of logits
        [n, vocab] (bf16, fp16 or fp32; rows may be strided slices) times scale,
        their lse and entropy [n], and the most likely tokens with theirs
        [n, top].  See kvr_token_logprobs."""
        here = _here()
        if getattr(logits, "ndim", 2) != 2:
            raise ValueError(f"logits: {logits.ndim} dimensions, the call needs [n, vocab]")
        kind = _typed(logits, "logits", _VALUE_TYPES, here)
        if logits.shape[0] != n:
            raise ValueError(f"logits: {logits.shape[0]} rows, the call has {n}")
        m = top = 0
        if (tokens is None) != (logprob is None) or (top_ids is None) != (top_logprob is None):
            raise ValueError("tokens go with logprob, and top_ids with top_logprob")
        if tokens is not None:
            if getattr(tokens, "ndim", 2) != 2:
                raise ValueError(f"tokens: {tokens.ndim} dimensions, the call needs [n, m]")
            shape = (n, int(tokens.shape[1]) if hasattr(tokens, "shape") else 0)
            m = shape[1]
            tokens = _full(tokens, "tokens", "int32", here, shape)
            logprob = _full(logprob, "logprob", "float32", here, shape)
        if top_ids is not None:
            if getattr(top_ids, "ndim", 2) != 2:
                raise ValueError(f"top_ids: {top_ids.ndim} dimensions, the call needs [n, top]")
            shape = (n, int(top_ids.shape[1]) if hasattr(top_ids, "shape") else 0)
            top = shape[1]
            top_ids = _full(top_ids, "top_ids", "int32", here, shape)
            top_logprob = _full(top_logprob, "top_logprob", "float32", here, shape)
        if lse is not None:
            lse = _full(lse, "lse", "float32", here, (n,))
        if entropy is not None:
            entropy = _full(entropy, "entropy", "float32", here, (n,))
        ws, ws_bytes = _workspace(workspace, here)
        call = LogprobCall(_VALUE_TYPES[kind], n, logits.shape[1], m, top, scale,
                           logits.data_ptr(), logits.stride(0), tokens, logprob, lse, entropy,
                           top_ids, top_logprob, ws, ws_bytes)
        _check(lib().kvr_token_logprobs(self.handle, ctypes.byref(call), _stream(stream, here)))

    # ------------------------------------------- pages shared by requests

    def bind_page_refs(self, refs):
        """int32 [pool_pages] map entries naming each physical page, or None."""
        _check(lib().kvr_bind_page_refs(self.handle, _words(refs, "refs", self.cfg.pool_pages)))

    def count_page_refs(self, stream=None):
        _check(lib().kvr_count_page_refs(self.handle, _stream(stream)))

    def release_requests(self, n, req_ids, status=None, stream=None):
        """Each listed request gives up its rows and pages.  What was resolved for
        it before must have run before it is set up again or forked into."""
        _check(lib().kvr_release_requests(self.handle, n, _words(req_ids, "req_ids", n),
                                          _words(status, "status", n), _stream(stream)))

    def fork_requests(self, n, src_ids, dst_ids, status=None, stream=None):
        """Request dst_ids[i] becomes a copy of src_ids[i].  The host fills of the
        source's last resolve may be outstanding; those of earlier ones, deferred
        appends and what was resolved for dst_ids[i] must have run."""
        _check(lib().kvr_fork_requests(self.handle, n, _words(src_ids, "src_ids", n),
                                       _words(dst_ids, "dst_ids", n),
                                       _words(status, "status", n), _stream(stream)))

    def copy_pages(self, n, req_ids, pages, phys, status, stream=None):
        _check(lib().kvr_copy_pages(self.handle, n, _words(req_ids, "req_ids", n),
                                    _words(pages, "pages", n), _words(phys, "phys", n),
                                    _words(status, "status", n), _stream(stream)))

    def pool_workspace(self) -> int:
        """Workspace bytes of list_free_pages and compact_pool."""
        got = lib().kvr_pool_workspace(self.handle)
        return got if got >= 0 else _check(got)

    def list_free_pages(self, free_list, free_count, workspace, stream=None):
        ws, ws_bytes = _workspace(workspace)
        _check(lib().kvr_list_free_pages(
            self.handle, _words(free_list, "free_list", self.cfg.pool_pages),
            _words(free_count, "free_count", 1), ws, ws_bytes, _stream(stream)))

    def compact_pool(self, max_moves, moves, move_count, workspace, stream=None):
        ws, ws_bytes = _workspace(workspace)
        need = 2 * max(0, min(max_moves, self.cfg.pool_pages))
        _check(lib().kvr_compact_pool(self.handle, max_moves, _words(moves, "moves", need),
                                      _words(move_count, "move_count", 1), ws, ws_bytes,
                                      _stream(stream)))


class Residency:
    """Host-side residency policy of one source's optional pool
    (kvr_residency_*): which pages to reclaim for an admission and which to
    refill.  Its decisions are applied with Context.reclaim_pages and
    Context.restore_pages."""

    def __init__(self, page_map, n_complete: int, pool_pages: int):
        import numpy as np
        pm = np.ascontiguousarray(page_map, dtype=np.int32)
        self.n_req, self.n_pages = pm.shape
        self.n_complete = int(n_complete)
        h = ctypes.c_void_p()
        _check(lib().kvr_residency_create(self.n_req, self.n_pages, self.n_complete,
                                          int(pool_pages), pm.ctypes.data, ctypes.byref(h)))
        self.handle = h.value

    def close(self):
        if self.handle:
            lib().kvr_residency_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def admit(self, need: int, order):
        """(True, [(request, page), ...] to reclaim, handle), or (False, [], -1)
        when the shortfall is larger than all optional pages together."""
        import numpy as np
        order = np.ascontiguousarray(order, dtype=np.int32)
        cap = self.n_req * self.n_complete
        req = np.zeros(max(1, cap), dtype=np.int32)
        page = np.zeros(max(1, cap), dtype=np.int32)
        n, h = ctypes.c_int32(), ctypes.c_int32()
        rc = lib().kvr_residency_admit(self.handle, int(need), len(order), order.ctypes.data, cap,
                                       req.ctypes.data, page.ctypes.data, ctypes.byref(n),
                                       ctypes.byref(h))
        if rc == E_CAPACITY:
            return False, [], -1
        _check(rc)
        return True, list(zip(req[:n.value].tolist(), page[:n.value].tolist())), h.value

    def release(self, handle: int):
        _check(lib().kvr_residency_release(self.handle, handle))

    def refill(self, bound: int):
        """[(request, page, physical page), ...] to restore."""
        import numpy as np
        cap = max(1, bound)
        req = np.zeros(cap, dtype=np.int32)
        page = np.zeros(cap, dtype=np.int32)
        phys = np.zeros(cap, dtype=np.int32)
        n = ctypes.c_int32()
        _check(lib().kvr_residency_refill(self.handle, bound, cap, req.ctypes.data,
                                          page.ctypes.data, phys.ctypes.data, ctypes.byref(n)))
        m = n.value
        return list(zip(req[:m].tolist(), page[:m].tolist(), phys[:m].tolist()))

    def counts(self):
        """(free pages, ready pages, reserved pages)."""
        f, r, s = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(lib().kvr_residency_counts(self.handle, ctypes.byref(f), ctypes.byref(r),
                                          ctypes.byref(s)))
        return f.value, r.value, s.value


class DraftRing:
    """Drafter visible-window ring (kvr_draft_*) over caller-owned device
    buffers: ring [n_req][capacity][row_bytes] (or None, with row_bytes 0, for a
    ring of K/V layers only), length and high int32 [n_req]."""

    def __init__(self, n_req, window, capacity, row_bytes, ring, length, high):
        h = ctypes.c_void_p()
        self.n_req, self.window_rows, self.row_bytes = n_req, window, row_bytes
        self.capacity, self.kv_heads, self.d_head = capacity, 0, 0
        _check(lib().kvr_draft_create(n_req, window, capacity, row_bytes,
                                      _dev(ring, "ring", max(n_req, 0) * max(capacity, 0) *
                                           max(row_bytes, 0)),
                                      _dev(length, "length", 4 * max(n_req, 0)),
                                      _dev(high, "high", 4 * max(n_req, 0)), ctypes.byref(h)))
        self.handle = h.value

    def close(self):
        if self.handle:
            lib().kvr_draft_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def reset(self, stream=None):
        _check(lib().kvr_draft_reset(self.handle, _stream(stream)))

    def append(self, n, req_ids, rows_each, rows, status=None, stream=None):
        need = max(n, 0) * max(rows_each, 0) * self.row_bytes
        _check(lib().kvr_draft_append(self.handle, n, _dev(req_ids, "req_ids", 4 * n), rows_each,
                                      _dev(rows, "rows", need), _dev(status, "status", 4 * n),
                                      _stream(stream)))

    def rollback(self, n, req_ids, keep, status=None, stream=None):
        _check(lib().kvr_draft_rollback(self.handle, n, _dev(req_ids, "req_ids", 4 * n),
                                        _dev(keep, "keep", 4 * n), _dev(status, "status", 4 * n),
                                        _stream(stream)))

    def window(self, n, req_ids, out, visible=None, status=None, stream=None):
        need = max(n, 0) * self.window_rows * self.row_bytes
        _check(lib().kvr_draft_window(self.handle, n, _dev(req_ids, "req_ids", 4 * n),
                                      _dev(out, "out", need), _dev(visible, "visible", 4 * n),
                                      _dev(status, "status", 4 * n), _stream(stream)))

    # ------------------------------------------- keys and values in 8 bits

    def bind_kv(self, n_layers, kv_heads, d_head, codes, scales):
        """K/V layers of the ring: codes (8-bit) [n_layers, n_req, capacity / 64,
        kv_heads, 2, 64 * d_head] and scales uint8 [n_layers, n_req,
        capacity / 64, kv_heads, 2].  See kvr_draft_bind_kv."""
        here = _here()
        units = max(n_layers, 0) * self.n_req * (self.capacity // DRAFT_BLOCK) * max(kv_heads, 0) * 2
        _check(lib().kvr_draft_bind_kv(
            self.handle, n_layers, kv_heads, d_head,
            _dev_here(codes, "codes", units * DRAFT_BLOCK * max(d_head, 0), here),
            _dev_here(scales, "scales", units, here)))
        self.kv_heads, self.d_head = kv_heads, d_head

    def write_kv(self, layer, n, req_ids, k, v, count=None, status=None, stream=None):
        """New tokens' keys and values [n, rows, kv_heads, d_head] (bf16, fp16 or
        fp32, one type; strided slices with contiguous heads) of a layer, at the
        positions after the rows kept; count int32 [n] of them (all, without it).
        See kvr_draft_write_kv."""
        here = _here()
        if getattr(k, "ndim", 4) != 4:
            raise ValueError(f"k: {k.ndim} dimensions, the call needs [n, rows, kv_heads, d_head]")
        kind = _typed(k, "k", _VALUE_TYPES, here)
        shape = (n, int(k.shape[1]), self.kv_heads, self.d_head)
        if k.shape != shape:
            _typed(k, "k", (kind,), here, shape)
        _typed(v, "v", (kind,), here, shape)
        ks, vs = k.stride(), v.stride()
        call = DraftWriteCall(layer, _VALUE_TYPES[kind], n, shape[1],
                              _words(req_ids, "req_ids", n, here),
                              _words(count, "count", n, here), k.data_ptr(), v.data_ptr(),
                              ks[0], ks[1], ks[2], vs[0], vs[1], vs[2],
                              _words(status, "status", n, here))
        _check(lib().kvr_draft_write_kv(self.handle, ctypes.byref(call), _stream(stream, here)))

    def read_kv(self, layer, n, req_ids, k, v, visible=None, status=None, stream=None):
        """The visible rows of a layer, oldest first, into k and v [n, window,
        kv_heads, d_head] (bf16, fp16 or fp32; rows past the window's length are
        untouched), their number into visible.  See kvr_draft_read_kv."""
        here = _here()
        shape = (n, self.window_rows, self.kv_heads, self.d_head)
        kind = _typed(k, "k", _VALUE_TYPES, here, shape)
        _check(lib().kvr_draft_read_kv(self.handle, layer, n, _words(req_ids, "req_ids", n, here),
                                       _VALUE_TYPES[kind], _full(k, "k", kind, here, shape),
                                       _full(v, "v", kind, here, shape),
                                       _words(visible, "visible", n, here),
                                       _words(status, "status", n, here), _stream(stream, here)))

    def advance(self, n, req_ids, rows, count=None, status=None, stream=None):
        """The tokens written to the K/V layers (count of each entry, or rows) become
        rows kept.  See kvr_draft_advance."""
        here = _here()
        _check(lib().kvr_draft_advance(self.handle, n, _words(req_ids, "req_ids", n, here), rows,
                                       _words(count, "count", n, here),
                                       _words(status, "status", n, here), _stream(stream, here)))

    def attend_workspace(self, n, nq, heads) -> int:
        """Workspace bytes for attend calls of up to these sizes."""
        got = lib().kvr_draft_attend_workspace(self.handle, n, nq, heads)
        return got if got >= 0 else _check(got)

    def attend(self, layer, n, req_ids, q, out, *, scale, mask="causal", count=None, lse=None,
               status=None, workspace=None, stream=None):
        """Attention of q [n, nq, heads, d_head] (bf16) over the window of a layer
        into out of that shape and lse [n, nq, heads]: each query sees the last
        window rows up to its own token ("causal"), up to the last new token
        ("block") or up to the last row kept ("kept").  See kvr_draft_attend."""
        here = _here()
        if getattr(q, "ndim", 4) != 4:
            raise ValueError(f"q: {q.ndim} dimensions, the call needs [n, nq, heads, d_head]")
        _typed(q, "q", ("bfloat16",), here)
        shape = (n, int(q.shape[1]), int(q.shape[2]), self.d_head)
        if q.shape != shape:
            _typed(q, "q", ("bfloat16",), here, shape)
        out = _full(out, "out", "bfloat16", here, shape)
        if lse is not None:
            lse = _full(lse, "lse", "float32", here, shape[:3])
        ws, ws_bytes = _workspace(workspace, here)
        qs = q.stride()
        call = DraftAttendCall(layer, _choice(mask, "mask", DRAFT_MASKS), n, shape[1], shape[2],
                               scale, _words(req_ids, "req_ids", n, here),
                               _words(count, "count", n, here), q.data_ptr(), qs[0], qs[1], qs[2],
                               out, lse, _words(status, "status", n, here), ws, ws_bytes)
        _check(lib().kvr_draft_attend(self.handle, ctypes.byref(call), _stream(stream, here)))


class StagingPool:
    """Verification staging reuse (kvr_staging_*): buffer indices handed out
    round-robin; acquire waits for the buffer's last release."""

    def __init__(self, n_buffers: int):
        h = ctypes.c_void_p()
        _check(lib().kvr_staging_create(n_buffers, ctypes.byref(h)))
        self.handle = h.value

    def close(self):
        if self.handle:
            lib().kvr_staging_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def acquire(self, stream=None) -> int:
        idx = ctypes.c_int32()
        _check(lib().kvr_staging_acquire(self.handle, _stream(stream), ctypes.byref(idx)))
        return idx.value

    def release(self, index: int, stream=None):
        _check(lib().kvr_staging_release(self.handle, index, _stream(stream)))
