"""Rotary positions against a plain 64-bit form.

Tolerances.  eps = 2^-24.  position * frequency and its whole turns are taken in
64 bits: the angle's fraction f is off by at most 2^31 2^-53 turns (positions
below 2^31, frequencies below 1/2) and by its rounding to 32 bits, 2^-25 turns of
|f| <= 1/2: the angle by 2 pi (2^-22 + |f| eps) <= 2^-19 at 2^31 and by 4 eps
below 2^22.  Sine and cosine of the library are within 4 eps, times the
magnitude one more: each factor is off by at most a = 12 eps (positions below
2^22) of the magnitude, the two products and their sum round three times: |y -
exact| <= (a + 4 eps) magnitude (|u| + |v|), then half a step of the type.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
TYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25),
        "f32": (2.0 ** -24, 2.0 ** -150)}
DEV = "cuda"


def context():
    from hierarchical_sparse_kv_resolve_amd import Context
    return Context(n_req=1, n_layers=1, history_rows=0, max_new_rows=1, page_rows=1, tail_rows=0,
                   hot_slots=1, row_bytes=16, sel_cap=1, pool_pages=0)


def frequencies(d_rot, base=10000.0):
    i = np.arange(d_rot // 2)
    return torch.from_numpy(base ** (-2.0 * i / d_rot) / (2 * math.pi)).to(DEV)


def check(y, x, positions, freq, d_rot, at, layout, magnitude, inverse, typ, far=12 * EPS):
    x, y, f = x.cpu().double().numpy(), y.cpu().double().numpy(), freq.cpu().numpy()
    # whole turns of position * frequency, split so that nothing is lost
    p = positions.cpu().numpy().astype(np.float64)
    hi = np.trunc(f * 2.0 ** 20) / 2.0 ** 20
    turns = np.mod(p[:, None] * hi, 1.0) + p[:, None] * (f - hi)
    a = 2 * np.pi * turns * (-1 if inverse else 1)
    c, s = magnitude * np.cos(a)[:, None], magnitude * np.sin(a)[:, None]
    part, got = x[..., at:at + d_rot], y[..., at:at + d_rot]
    pick = (lambda z: (z[..., :d_rot // 2], z[..., d_rot // 2:])) if layout == "half" else \
        (lambda z: (z[..., 0::2], z[..., 1::2]))
    u, v = pick(part)
    gu, gv = pick(got)
    half, tiny = HALF[typ]
    slack = (far + 4 * EPS) * abs(magnitude) * (np.abs(u) + np.abs(v))
    for g, w in ((gu, u * c - v * s), (gv, v * c + u * s)):
        assert (np.abs(g - w) <= slack + half * (np.abs(w) + slack) + tiny).all()
    rest = np.delete(x, np.s_[at:at + d_rot], axis=-1)
    assert np.array_equal(np.delete(y, np.s_[at:at + d_rot], axis=-1), rest)


@pytest.mark.parametrize("typ", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("d_head,at,d_rot", [(128, 0, 128), (576, 512, 64), (128, 32, 96),
                                             (64, 0, 16), (80, 0, 20), (67, 3, 6), (70, 1, 2),
                                             (1024, 0, 1024)])
@pytest.mark.parametrize("n,heads,kheads", [(1, 1, 0), (3, 16, 1), (150, 5, 2)])
def test_rotate(typ, layout, d_head, at, d_rot, n, heads, kheads):
    rng = np.random.default_rng(n + d_head)
    make = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(TYPE[typ]).to(DEV)  # noqa: E731
    q, k = make(n, heads, d_head), make(n, kheads, d_rot) if kheads else None
    pos = torch.from_numpy(rng.integers(0, 1 << 20, n).astype(np.int32)).to(DEV)
    pos[0] = 0
    freq = frequencies(d_rot)
    x = context()
    for magnitude, inverse in ((1.0, False), (1.25, True)):
        out = torch.full_like(q, 7.0)
        kout = torch.full_like(k, 7.0) if kheads else None
        kw = dict(d_rot=d_rot, layout=layout, at=at, magnitude=magnitude, inverse=inverse)
        x.rotate_rows(n, pos, freq, q, out, k, kout, **kw)
        check(out, q, pos, freq, d_rot, at, layout, magnitude, inverse, typ)
        if kheads:
            check(kout, k, pos, freq, d_rot, 0, layout, magnitude, inverse, typ)
        own, kown = q.clone(), None if k is None else k.clone()
        x.rotate_rows(n, pos, freq, own, key=kown, **kw)  # in place
        assert torch.equal(own, out) and (k is None or torch.equal(kown, kout))


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("typ", ["bf16", "f32"])
@pytest.mark.parametrize("first", [0, 8, 1, 3])
def test_slices(layout, typ, first):
    """Heads as slices of a wider tensor (aligned or not), tokens of a larger batch,
    one tensor's rows for all; what lies beside them stays."""
    wide = torch.randn(40, 3, 220, device=DEV).to(TYPE[typ])
    before = wide.clone()
    x = wide[::2, :, first:first + 192]
    pos = torch.randint(0, 5000, (20,), dtype=torch.int32, device=DEV)
    freq = frequencies(64)
    out = torch.zeros(20, 3, 192, device=DEV, dtype=TYPE[typ])
    c = context()
    kw = dict(d_rot=64, layout=layout, at=128)
    c.rotate_rows(20, pos, freq, x, out, **kw)
    check(out, x, pos, freq, 64, 128, layout, 1.0, False, typ)
    assert torch.equal(wide, before)
    c.rotate_rows(20, pos, freq, x, **kw)
    assert torch.equal(x, out)
    x.copy_(before[::2, :, first:first + 192])
    assert torch.equal(wide, before)
    one = before[:1, :, first:first + 192].expand(20, 3, 192)
    c.rotate_rows(20, pos, freq, one, out, **kw)
    check(out, one, pos, freq, 64, 128, layout, 1.0, False, typ)


def test_key_alone():
    k = torch.randn(9, 1, 64, device=DEV)
    pos = torch.arange(9, dtype=torch.int32, device=DEV)
    out = torch.zeros_like(k)
    context().rotate_rows(9, pos, frequencies(64), None, None, k, out, d_rot=64, layout="half")
    check(out, k, pos, frequencies(64), 64, 0, "half", 1.0, False, "f32")


def test_far_and_negative_positions():
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 2 ** 24 + 1, 2 ** 30 + 3], dtype=torch.int32,
                       device=DEV)
    x = torch.randn(5, 2, 128, device=DEV)
    out = torch.zeros_like(x)
    freq = frequencies(128)
    context().rotate_rows(5, pos, freq, x, out, d_rot=128, layout="half")
    check(out, x, pos, freq, 128, 0, "half", 1.0, False, "f32", far=2.0 ** -18)


def test_turning_back():
    """The inverse takes positions off again; it is the gradient of the rotation."""
    x = torch.randn(33, 4, 128, device=DEV, dtype=torch.float32)
    g = torch.randn_like(x)
    pos = torch.randint(0, 100000, (33,), dtype=torch.int32, device=DEV)
    freq = frequencies(64)
    c = context()
    kw = dict(d_rot=64, layout="interleaved", at=32, magnitude=1.5)
    y, back, grad = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    c.rotate_rows(33, pos, freq, x, y, **kw)
    c.rotate_rows(33, pos, freq, y, back, **{**kw, "magnitude": 1 / 1.5}, inverse=True)
    # twice the error above, of values of at most the pair's size
    size = x.abs().amax(-1, keepdim=True) * 2
    assert ((back - x).abs() <= 2 * 16 * EPS * 2 * size).all()
    c.rotate_rows(33, pos, freq, g, grad, **kw, inverse=True)
    # <R x, g> = <x, R^T g>, for the rotated part and the rest
    a, b = (y.double() * g.double()).sum(), (x.double() * grad.double()).sum()
    assert abs(a - b) <= 16 * EPS * 2 * (y.double().abs() * g.double().abs()).sum() * 2
    # and differences of the loss <R x, g>
    e = torch.zeros_like(x)
    e[5, 2, 40] = 1.0
    y2 = torch.zeros_like(x)
    c.rotate_rows(33, pos, freq, x + e, y2, **kw)
    slope = ((y2 - y).double() * g.double()).sum()
    bound = 64 * EPS * (y.double().abs() * g.double().abs())[5, 2].sum() + 64 * EPS * g[5, 2].abs().sum() * 4
    assert abs(slope - grad[5, 2, 40]) <= bound


def test_many_tokens_and_past_32_bits():
    """A tensor of more than 4 GiB: its last tokens, and the first."""
    n, heads, d = 40000, 110, 512
    x = torch.empty(n, heads, d, dtype=torch.bfloat16, device=DEV)
    assert x.numel() * 2 > 4 << 30
    ends = torch.tensor([0, 1, 17, n // 2, n - 2, n - 1], device=DEV)
    x[ends] = torch.randn(6, heads, d, device=DEV).bfloat16()
    src = x[ends].clone()
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    freq = frequencies(64)
    context().rotate_rows(n, pos, freq, x, d_rot=64, layout="half", at=448)
    check(x[ends], src, pos[ends], freq, 64, 448, "half", 1.0, False, "bf16")


def test_other_stream_and_graph():
    x = torch.randn(64, 16, 128, device=DEV).bfloat16()
    pos = torch.randint(0, 9999, (64,), dtype=torch.int32, device=DEV)
    freq, out, want = frequencies(128), torch.zeros_like(x), torch.zeros_like(x)
    c = context()
    kw = dict(d_rot=128, layout="half")
    c.rotate_rows(64, pos, freq, x, want, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.rotate_rows(64, pos, freq, x, out, **kw, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.rotate_rows(64, pos, freq, x, out, **kw)
    for _ in range(3):
        x.copy_(torch.randn_like(x, dtype=torch.float32))
        pos.copy_(torch.randint(0, 9999, (64,), device=DEV))
        g.replay()
        c.rotate_rows(64, pos, freq, x, want, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_launch_timing_and_no_work():
    c = context()
    x = torch.randn(2, 1, 64, device=DEV)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    c.timing_begin(8)
    c.rotate_rows(2, pos, frequencies(64), x, d_rot=64, layout="half")
    c.rotate_rows(0, pos[:0], frequencies(64), x[:0], d_rot=64, layout="half")
    assert [k for k, _ in c.timing_end()] == ["rotate"]


def test_refusals():
    from hierarchical_sparse_kv_resolve_amd import KvrError
    c = context()
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    good = dict(n=4, positions=pos, frequencies=frequencies(64), x=x, d_rot=64, layout="half", at=64)
    c.rotate_rows(**good)

    def refused(error, match, **kw):
        with pytest.raises(error, match=match):
            c.rotate_rows(**{**good, **kw})

    refused(ValueError, "unknown layout", layout="neox")
    refused(KvrError, r"values \[65, 129\) are not in a head of 128", at=65)
    refused(KvrError, "not in a head", at=-1)
    refused(KvrError, "d_rot must be even", d_rot=3, frequencies=frequencies(2))
    refused(ValueError, "frequencies: shape", d_rot=32)
    refused(TypeError, "frequencies: expected float64", frequencies=frequencies(64).float())
    refused(TypeError, "positions: expected int32", positions=pos.long())
    refused(ValueError, "positions: ", positions=pos[:3])
    refused(ValueError, "x: 4 tokens", n=3)
    refused(ValueError, "dimensions", x=x[0])
    refused(TypeError, "GPU tensor", x=x.cpu())
    refused(TypeError, "x's output: expected bfloat16", out=x.float())
    refused(ValueError, "x's output: shape", out=x[:, :1])
    refused(TypeError, "key: expected bfloat16", key=x.half())
    refused(ValueError, "an output without an input", key_out=x)
    refused(ValueError, "x or key", x=None)
    refused(ValueError, "last dimension",
            x=torch.zeros(4, 128, 2, dtype=torch.bfloat16, device=DEV).transpose(1, 2))
    one = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device=DEV).expand(4, 2, 128)
    refused(KvrError, "an output stride of 0", x=one)
    refused(KvrError, "an output stride of 0", out=one)
    refused(KvrError, "key: an output stride of 0", key=one)
    with pytest.raises(KvrError, match="same strides"):
        c.rotate_rows(**{**good, "out": x.view(-1)[:4 * 2 * 128].as_strided((4, 2, 128),
                                                                          (128, 512, 1))})
