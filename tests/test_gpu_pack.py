"""Packing of rows against a plain 64-bit form.

Tolerances.  e = 2^-24.  The sum of squares of d_v values is a tree of at most
d_v / 64 + 6 roundings on top of each product's one, the mean, the addition of
eps, the square root and the reciprocal round once each and count half in the
root: 1/sqrt is off by at most ((d_v / 64 + 8) / 2 + 3) e relative; the two
products by it and the weight add 2 e.  x is therefore off by at most X = 12 e
(relative, d_v up to 512).  16-bit rows: X |x| + half a step of the type (a value
below fp16's normal range: half of 2^-24).  fp8 scales: X + e.  A code is
e4m3(x / scale) with x / scale off by at most (2 X + 3 e) relative: the value code
* scale is within half an e4m3 step (2^-4 relative, 2^-10 below the smallest
normal 2^-6) of x / scale, times the scale, plus that error.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import attend_reference as ref

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
X = 12 * E
SRC = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def context(fmt, d_v, d_rope):
    from hierarchical_sparse_kv_resolve_amd import Context
    return Context(n_req=1, n_layers=1, history_rows=0, max_new_rows=1, page_rows=1, tail_rows=0,
                   hot_slots=1, row_bytes=ref.row_bytes(fmt, d_v, d_rope), sel_cap=1, pool_pages=0)


def pack(fmt, d_v, d_rope, latent, rope, weight=None, eps=0.0, rows=None):
    n = latent.shape[0]
    R = ref.row_bytes(fmt, d_v, d_rope)
    if rows is None:
        rows = torch.full((n + 1, R), 0xA5, dtype=torch.uint8, device="cuda")
    context(fmt, d_v, d_rope).pack_rows(n, latent, rope, rows, fmt=fmt, d_v=d_v, d_rope=d_rope,
                                        weight=weight, eps=eps)
    torch.cuda.synchronize()
    assert (rows[n:] == 0xA5).all(), "a row past the last was written"
    return rows[:n].cpu()


def check(rows, fmt, d_v, d_rope, latent, rope, weight=None, eps=0.0):
    x = latent.cpu().double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * weight.cpu().double()
    typ = ref.TYPE[fmt]
    half, tiny = (2.0 ** -11, 2.0 ** -25) if fmt == "f16" else (2.0 ** -8, 2.0 ** -134)
    if d_rope:
        # one rounding of the given value
        got = rows[:, rows.shape[1] - 2 * d_rope:].contiguous().view(typ)
        assert torch.equal(got, rope.cpu().to(typ))
    if fmt != "fp8":
        got = rows[:, :2 * d_v].contiguous().view(typ).double()
        assert ((got - x).abs() <= (X + half) * x.abs() * (1 + X) + tiny).all()
        return
    groups = d_v // 128
    top = x.view(-1, groups, 128).abs().amax(2)
    want = torch.where(top == 0, 1.0, top / 448)
    raw = rows[:, d_v:d_v + (groups * 4 + 15) // 16 * 16].contiguous()
    scale = raw[:, :4 * groups].contiguous().view(torch.float32).double()
    assert (raw[:, 4 * groups:] == 0).all(), "the padding of the scales"
    assert ((scale - want).abs() <= (X + E) * want + 2.0 ** -149).all()
    code = rows[:, :d_v].contiguous().view(torch.float8_e4m3fn).double()
    ratio = x / want.repeat_interleave(128, 1)
    err = (code - ratio).abs()
    slack = (2 * X + 3 * E) * ratio.abs()
    assert (err <= (2.0 ** -4 * (ratio.abs() + slack)).clamp(min=2.0 ** -10) + slack).all()


FORMATS = [("fp8", 512, 64), ("bf16", 512, 64), ("f16", 512, 64), ("fp8", 256, 64), ("fp8", 512, 0),
           ("f16", 256, 0)]


@pytest.mark.parametrize("fmt,d_v,d_rope", FORMATS)
@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [1, 3, 130])
@pytest.mark.parametrize("norm", [True, False])
def test_pack(fmt, d_v, d_rope, src, n, norm):
    rng = np.random.default_rng(n + 7 * norm)
    latent = torch.from_numpy(rng.standard_normal((n, d_v)) * np.exp(rng.standard_normal((n, 1))))
    latent = latent.to(SRC[src]).cuda()
    rope = torch.from_numpy(rng.standard_normal((n, d_rope))).to(SRC[src]).cuda()
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(d_v)).float().cuda() if norm else None
    rows = pack(fmt, d_v, d_rope, latent, rope, w, 1e-6)
    check(rows, fmt, d_v, d_rope, latent, rope, w, 1e-6)


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("width,at", [(576, 0), (640, 64), (577, 1), (579, 3)])
@pytest.mark.parametrize("src", ["bf16", "f32"])
def test_slices_of_one_projection(fmt, width, at, src):
    """Latent and rope part as slices of one tensor, at any element offset."""
    rng = np.random.default_rng(3)
    both = torch.from_numpy(rng.standard_normal((37, width))).to(SRC[src]).cuda()
    latent, rope = both[:, at:at + 512], both[:, at + 512:at + 576]
    w = torch.ones(512, device="cuda")
    check(pack(fmt, 512, 64, latent, rope, w, 1e-6), fmt, 512, 64, latent, rope, w, 1e-6)


def test_one_row_for_all():
    """A row stride of 0 packs one token n times."""
    latent = torch.randn(1, 512, device="cuda").expand(9, 512)
    rope = torch.randn(1, 64, device="cuda").expand(9, 64)
    rows = pack("fp8", 512, 64, latent, rope)
    check(rows, "fp8", 512, 64, latent, rope)
    assert (rows == rows[0]).all()


def test_zeros_and_extremes():
    """Rows and groups of zeros, one spike, sizes near both ends of the range."""
    x = torch.zeros(6, 512)
    x[1, 130] = 3.0
    x[2] = torch.linspace(-1, 1, 512) * 1e-30
    x[3] = torch.linspace(-1, 1, 512) * 1e30
    x[4, :128] = 1e-38
    x[5] = torch.linspace(0, 448, 512)
    x, rope = x.cuda(), torch.zeros(6, 64).cuda()
    check(pack("fp8", 512, 64, x, rope), "fp8", 512, 64, x, rope)
    y = x[[0, 1, 5]]
    w = torch.ones(512, device="cuda")
    check(pack("fp8", 512, 64, y, rope[:3], w, 1e-6), "fp8", 512, 64, y, rope[:3], w, 1e-6)


def test_norm_past_the_32_bit_range():
    """A row whose squares overflow 32 bits becomes 0, its neighbours keep theirs."""
    latent = torch.randn(3, 512, device="cuda")
    latent[1] *= 1e20
    rope, w = torch.zeros(3, 64, device="cuda"), torch.ones(512, device="cuda")
    got = ref.unpack(pack("bf16", 512, 64, latent, rope, w, 1e-6), "bf16", 512, 64)
    assert (got[1] == 0).all()
    keep = pack("bf16", 512, 64, latent[[0, 2]], rope[[0, 2]], w, 1e-6)
    assert torch.equal(got[[0, 2]], ref.unpack(keep, "bf16", 512, 64))


@pytest.mark.parametrize("d_v", [512, 256])
@pytest.mark.parametrize("norm", [False, True])
def test_groups_of_subnormal_scale(d_v, norm):
    """Groups whose largest value is u steps of 2^-149: the scale u / 448 steps
    rounds to whole steps (to none below 224, a group of zeros then) and the
    quotient may exceed the largest code.  Every code is finite, and a value is
    off by half a step of its code, or by what the largest code times the scale
    cannot reach, 448 times half a step of the scale; a NaN stays in its group."""
    step = 2.0 ** -149
    tops = [1, 3, 200, 223, 225, 300, 447, 448, 500, 627, 671, 673, 700, 1000, 2000, 5000, 1 << 16,
            1 << 22]
    rng = np.random.default_rng(8)
    groups = d_v // 128
    u = np.array([[tops[(i + g) % len(tops)] for g in range(groups)] for i in range(len(tops))])
    x = np.floor(rng.random((len(tops), groups, 128)) * (u[..., None] + 1))
    x[:, :, 5] = u
    x = torch.from_numpy(x * np.where(rng.random(x.shape) < 0.5, -1, 1)).view(len(tops), d_v)
    latent, w = (x * step).float().cuda(), None
    assert torch.equal(latent.cpu().double(), x * step)
    if norm:  # latents of 1 and such weights: one product each, the same for all rows
        x = x[9:10].expand(len(tops), d_v)
        latent, w = torch.ones(len(tops), d_v, device="cuda"), (x[0] * step).float().cuda()
    rope = torch.zeros(len(tops), 64, device="cuda")
    rows = pack("fp8", d_v, 64, latent, rope, w, 0.0)
    got = ref.unpack(rows, "fp8", d_v, 64)[:, :d_v] / step
    assert got.isfinite().all()
    top = x.reshape(len(tops), groups, 128).abs().amax(2).repeat_interleave(128, 1)
    # half a code's step (2^-4 relative; 2^-10 of the scale for the smallest codes), the rest
    tol = 2.0 ** -4 * x.abs() + 2.0 ** -10 * (top / 448 + 0.5) + 448 * 0.5
    assert ((got - x).abs() <= tol).all()
    if not norm:
        latent[9, 7] = float("nan")
        bad = ref.unpack(pack("fp8", d_v, 64, latent, rope), "fp8", d_v, 64)[:, :d_v] / step
        assert not bad[9, :128].isfinite().any()
        bad[9, :128] = got[9, :128]
        assert torch.equal(bad, got)


def test_nan_and_infinity_stay_in_their_group():
    x = torch.randn(3, 512)
    y = x.clone()
    y[0, 200], y[1, 511] = float("nan"), float("inf")
    rope = torch.randn(3, 64).cuda()
    good = ref.unpack(pack("fp8", 512, 64, x.cuda(), rope), "fp8", 512, 64)
    bad = ref.unpack(pack("fp8", 512, 64, y.cuda(), rope), "fp8", 512, 64)
    assert not bad[0, 128:256].isfinite().any() and not bad[1, 384:512].isfinite().any()
    good[0, 128:256] = bad[0, 128:256] = 0
    good[1, 384:512] = bad[1, 384:512] = 0
    assert torch.equal(good, bad)
    got = pack("bf16", 512, 64, y.cuda(), rope)[:, :1024].contiguous().view(torch.bfloat16)
    assert got[0, 200].isnan() and got[1, 511] == float("inf")
    assert int((~got.isfinite()).sum()) == 2


def test_rows_in_pinned_memory():
    """Imported rows go straight to a host store."""
    rng = np.random.default_rng(5)
    latent = torch.from_numpy(rng.standard_normal((200, 512))).bfloat16().cuda()
    rope = torch.from_numpy(rng.standard_normal((200, 64))).bfloat16().cuda()
    host = torch.full((201, 656), 0xA5, dtype=torch.uint8).pin_memory()
    rows = pack("fp8", 512, 64, latent, rope, rows=host)
    assert torch.equal(rows, pack("fp8", 512, 64, latent, rope))


def test_many_rows():
    """More rows than one grid's waves."""
    n = 70001
    latent = torch.randn(n, 512, device="cuda").bfloat16()
    rope = torch.randn(n, 64, device="cuda").bfloat16()
    w = torch.ones(512, device="cuda")
    check(pack("fp8", 512, 64, latent, rope, w, 1e-5), "fp8", 512, 64, latent, rope, w, 1e-5)


def test_captured_and_replayed():
    latent = torch.randn(50, 512, device="cuda").bfloat16()
    rope = torch.randn(50, 64, device="cuda").bfloat16()
    rows = torch.zeros(50, 656, dtype=torch.uint8, device="cuda")
    ctx = context("fp8", 512, 64)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        ctx.pack_rows(50, latent, rope, rows, fmt="fp8", d_v=512, d_rope=64)
    for _ in range(3):
        latent.copy_(torch.randn(50, 512, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(rows.cpu(), pack("fp8", 512, 64, latent, rope))


def test_refusals():
    from hierarchical_sparse_kv_resolve_amd import KvrError
    ctx = context("fp8", 512, 64)
    latent = torch.zeros(4, 512, device="cuda")
    rope = torch.zeros(4, 64, device="cuda")
    rows = torch.zeros(4, 656, dtype=torch.uint8, device="cuda")
    good = dict(n=4, latent=latent, rope=rope, rows=rows, fmt="fp8", d_v=512, d_rope=64)
    ctx.pack_rows(**good)
    ctx.pack_rows(**{**good, "n": 0, "latent": latent[:0], "rope": rope[:0]})
    for error, match, kw in (
            (ValueError, "unknown row format", dict(fmt="int8")),
            (TypeError, "latent: expected", dict(latent=latent.double())),
            (TypeError, "latent: expected a GPU tensor", dict(latent=latent.cpu())),
            (ValueError, "latent: shape", dict(latent=latent[:3])),
            (TypeError, "rope: expected float32", dict(rope=rope.half())),
            (TypeError, "rope: expected a GPU tensor", dict(rope=None)),
            (ValueError, "last dimension", dict(latent=torch.zeros(512, 4, device="cuda").T)),
            (TypeError, "weight: expected float32", dict(weight=torch.ones(512, device="cuda").half())),
            (ValueError, "weight: shape", dict(weight=torch.ones(256, device="cuda"))),
            (ValueError, "rows: 1968 bytes", dict(rows=rows[:3])),
            (TypeError, "pinned", dict(rows=rows.cpu())),
            (KvrError, "the context's have 656", dict(fmt="bf16")),
            (KvrError, "d_v is 256 or 512", dict(d_v=384, latent=latent[:, :384])),
            (KvrError, "not aligned", dict(rows=torch.zeros(4 * 656 + 16, dtype=torch.uint8,
                                                            device="cuda")[8:]))):
        with pytest.raises(error, match=match):
            ctx.pack_rows(**{**good, **kw})
