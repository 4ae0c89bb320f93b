"""Host-side checks, without a GPU, of rotation, log probabilities and the drafter's
K/V calls: null handles, sizes, the call structs' layout, the frequencies."""
from __future__ import annotations

import ctypes
import math
import os
import re

import numpy as np
import pytest

from hierarchical_sparse_kv_resolve_amd import kvr
from tests import draft_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kvr.h")).read(), flags=re.S)


def test_null_handles_and_calls():
    lib = kvr.lib()
    for name, args in (("kvr_rotate_rows", (ctypes.byref(kvr.RotateCall()), None)),
                       ("kvr_token_logprobs", (ctypes.byref(kvr.LogprobCall()), None))):
        assert getattr(lib, name)(None, *args) == kvr.E_ARG
        assert "null context" in kvr.last_error()
    for name, args in (("kvr_draft_bind_kv", (1, 1, 64, 16, 16)),
                       ("kvr_draft_write_kv", (ctypes.byref(kvr.DraftWriteCall()), None)),
                       ("kvr_draft_read_kv", (0, 0, None, 0, None, None, None, None, None)),
                       ("kvr_draft_advance", (0, None, 0, None, None, None)),
                       ("kvr_draft_attend", (ctypes.byref(kvr.DraftAttendCall()), None))):
        assert getattr(lib, name)(None, *args) == kvr.E_ARG, name
        assert "null drafter ring" in kvr.last_error()
    assert lib.kvr_draft_attend_workspace(None, 1, 1, 1) == kvr.E_ARG


def test_call_structs_match_the_header():
    c_types = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float,
               "size_t": ctypes.c_size_t, "kvr_rotate_part": kvr.RotatePart}
    for struct, cls in (("kvr_rotate_part", kvr.RotatePart), ("kvr_rotate_call", kvr.RotateCall),
                        ("kvr_logprob_call", kvr.LogprobCall),
                        ("kvr_draft_write_call", kvr.DraftWriteCall),
                        ("kvr_draft_attend_call", kvr.DraftAttendCall)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), HEADER,
                         re.S).group(1)
        want = []
        for line in filter(None, (x.strip() for x in body.split(";"))):
            name = re.search(r"(\w+)$", line).group(1)
            want.append((name, ctypes.c_void_p if "*" in line else c_types[line.split()[0]]))
        assert want == list(cls._fields_), struct


def test_choices_match_the_header():
    def enum(prefix):
        return {n.lower(): int(v) for n, v in re.findall(prefix + r"_([A-Z0-9]+)\s*=\s*(\d+)",
                                                         HEADER)}
    assert {k: v for k, v in enum("KVR_ROPE").items() if k in kvr.ROPE_LAYOUTS} == kvr.ROPE_LAYOUTS
    assert {k: v for k, v in enum("KVR_ROPE").items() if k not in kvr.ROPE_LAYOUTS} == \
        kvr.ROPE_SCALINGS
    assert enum("KVR_DRAFT") == {"causal": kvr.DRAFT_MASKS["causal"],
                                 "whole": kvr.DRAFT_MASKS["block"],
                                 "kept": kvr.DRAFT_MASKS["kept"]}
    assert f"#define KVR_DRAFT_BLOCK {kvr.DRAFT_BLOCK}" in HEADER


@pytest.mark.parametrize("n,vocab", [(-1, 10), (1, 0), (1, (1 << 24) + 1), ((1 << 20) + 1, 10)])
def test_logprob_workspace_refuses(n, vocab):
    with pytest.raises(kvr.KvrError):
        kvr.Context.logprob_workspace(n, vocab)


def test_logprob_workspace_covers_smaller_calls():
    size = kvr.Context.logprob_workspace
    for N, V in ((300, 131072), (1, 131072), (5000, 3000), (1024, 2049)):
        most = size(N, V)
        for n in {0, 1, 2, 7, 63, 300, 1000, 1023, 1024, 1025, 5000} & set(range(N + 1)) | {N}:
            for v in (1, 8, 2048, 2049, 3000, 50000, 131072):
                if v <= V:
                    assert 0 <= size(n, v) <= most


def test_unknown_names():
    with pytest.raises(ValueError, match="unknown scaling 'ntk': one of none, linear"):
        kvr.rope_frequencies(64, scaling="ntk")
    with pytest.raises(ValueError, match="unknown mask"):
        kvr._choice("full", "mask", kvr.DRAFT_MASKS)


@pytest.mark.parametrize("kw,match", [
    (dict(d_rot=7), "d_rot must be even"), (dict(d_rot=0), "d_rot must be even"),
    (dict(d_rot=2048), "d_rot must be even"), (dict(d_rot=8, base=1.0), "base must be above 1"),
    (dict(d_rot=8, base=float("nan")), "base must be above 1"),
    (dict(d_rot=8, factor=0.5), "factor at least 1"),
    (dict(d_rot=2, scaling="base", factor=2.0), "d_rot of 4"),
    (dict(d_rot=8, scaling="ramp", factor=2.0), "original_length"),
    (dict(d_rot=8, scaling="ramp", factor=2.0, original_length=9, beta_fast=1.0, beta_slow=1.0),
     "beta_fast > beta_slow"),
])
def test_frequencies_refuse(kw, match):
    with pytest.raises(kvr.KvrError, match=match):
        kvr.rope_frequencies(**kw)


def test_frequencies():
    """Each kind by its formula, in Python floats (64 bits: a few steps apart)."""
    d, base, s = 64, 10000.0, 16.0
    plain = [base ** (-2 * i / d) / (2 * math.pi) for i in range(d // 2)]

    def close(got, want):
        return np.allclose(got, want, rtol=1e-14, atol=0)

    f, m = kvr.rope_frequencies(d)
    assert close(f, plain) and m == 1.0
    f, m = kvr.rope_frequencies(d, scaling="linear", factor=s)
    assert close(f, [x / s for x in plain]) and m == 1.0
    f, m = kvr.rope_frequencies(d, scaling="base", factor=s)
    b = base * s ** (d / (d - 2))
    assert close(f, [b ** (-2 * i / d) / (2 * math.pi) for i in range(d // 2)]) and m == 1.0
    assert math.isclose(f[-1], plain[-1] / s, rel_tol=1e-12) and f[0] == plain[0]
    L = 4096
    f, m = kvr.rope_frequencies(d, scaling="ramp", factor=s, original_length=L)
    pair = lambda t: d * math.log(L / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
    low, high = math.floor(pair(32)), math.ceil(pair(1))
    want = []
    for i, x in enumerate(plain):
        r = min(max((i - low) / (high - low), 0), 1)
        want.append(x * (1 - r) + x / s * r)
    assert close(f, want) and math.isclose(m, 0.1 * math.log(s) + 1, rel_tol=1e-6)
    # pairs that turn often stay, slow ones are stretched in full
    assert f[0] == plain[0] and math.isclose(f[-1], plain[-1] / s, rel_tol=1e-14)
    # a context so short that no pair turns beta_fast times: the bounds hold
    f, _ = kvr.rope_frequencies(8, scaling="ramp", factor=2.0, original_length=2)
    assert np.isfinite(f).all() and (f > 0).all()


def test_plain_window():
    """The plain form itself: minimal scales, values within half a step, the ring."""
    rng = np.random.default_rng(0)
    w = ref.Window(1, 100, 128, 1, 64)
    kept = {}
    for step in range(300):
        x = rng.standard_normal((1, 1, 64)) * 2.0 ** rng.integers(-3, 4)
        x = x.astype(np.float32).astype(np.float64)
        w.write(0, x, 2 * x)
        w.advance(0, 1)
        kept[step] = x[0, 0]
    k, v = w.rows(0, 200, 300)
    for j in range(100):
        want = kept[200 + j]
        # a token is rounded at most once to normal codes; each scale it has seen may
        # have cut it to half of that scale's last step (2^-10 of at most 2^0)
        assert (np.abs(k[0, j] - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10)).all()
    for b in range(2):
        for i, part in enumerate((w.code[0], w.code[1])):
            top = np.abs(ref.values_of(part[0, 0, b * 64:(b + 1) * 64])).max()
            assert 224 < top <= 448 or w.exp[0, b, 0, i] == -100
    assert ref.exponent_for(448.0) == 0 and ref.exponent_for(np.nextafter(448.0, 999)) == 1
    assert ref.exponent_for(0.0) == -100 and ref.exponent_for(2.0 ** -200) == -100
