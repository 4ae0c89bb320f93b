"""Attention whose workgroups walk many tiles of 64 rows: the rotation of two
and of three tile buffers, words and map entries fetched ahead inside the loop,
and sums that are scaled down when a later tile exceeds their reference.

The calls have so many query rows that a selection is not cut into shares: a
workgroup walks all of it.  That a call launched one kernel (a cut one is
joined by a second) is asserted, so every call walks ceil(rows / 64) tiles.

Tolerances are those of test_gpu_attend (`check`).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import attend_reference as ref
from tests.test_gpu_attend import EPS32, HALF, Source, check, to_dev

pytestmark = pytest.mark.gpu

# both kinds of 16-bit rows and fp8 rows, with two tile buffers (16-bit rows of
# 512 values) and with three
FORMATS = [("bf16", 512, 64), ("fp8", 512, 64), ("f16", 512, 0), ("f16", 256, 64),
           ("fp8", 256, 0), ("bf16", 256, 0)]
# n, nq, heads, with a map: 130 to 132 blocks of up to 16 query rows, or of 32
SHAPES = {"16": (130, 2, 7, False), "16-map": (10, 13, 11, True), "32": (2, 3, 700, False),
          "32-map": (5, 13, 33, True)}
ROWS = {3: 150, 4: 256, 5: 257, 7: 400, 30: 1901}  # by tiles


def random_rows(rng, count, fmt, d_v, d_rope):
    """Distinct rows for up to 4096, then the same again in another order."""
    some = ref.random_rows(rng, min(count, 4096), fmt, d_v, d_rope)
    return some[torch.from_numpy(rng.permutation(count) % some.shape[0])]


def counts(n, stride):
    """None, one, a tile and its neighbours, parts, all and more."""
    kinds = [stride, 0, 1, 64, 65, 127, 129, stride - 1, stride // 2, stride + 9, -2]
    return [kinds[i % len(kinds)] for i in range(n)]


def some(n):
    """The entries that a call of many is checked at (each kind of count among them)."""
    return list(range(0, n, 3)) if n > 100 else list(range(n))


def attend(src, n, nq, heads, stride, q, scale, *, words=None, rows=None, count=None, map_=None,
           shares=False):
    """out, lse and status of one call; without `shares` it has to be one kernel."""
    typ = ref.TYPE[src.fmt]
    out = torch.full((n, nq, heads, src.d_v), 7.0, dtype=typ, device="cuda")
    lse = torch.full((n, nq, heads), 7.0, device="cuda")
    status = torch.zeros(n, dtype=torch.int32, device="cuda")
    k = stride if map_ is None else map_.shape[2]
    need = src.ctx.attend_workspace(n, nq, heads, src.d_v, k)
    ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    src.ctx.timing_begin(4)
    src.ctx.attend_rows(0, n, None, q, out, fmt=src.fmt, d_v=src.d_v, d_rope=src.d_rope, scale=scale,
                        stride=stride, loc=None if words is None else to_dev(words), rows=rows,
                        count=None if count is None else torch.tensor(count, dtype=torch.int32,
                                                                      device="cuda"),
                        map_=map_, lse=lse, status=status, workspace=ws)
    torch.cuda.synchronize()
    launches = len(src.ctx.timing_end())
    assert shares or launches == 1, "the selection was cut into shares"
    assert (ws[need:] == 0x7F).all()
    return out, lse, status


def keys_by_query(src, entries, nq, stride, *, words=None, rows=None, count=None, map_=None):
    """lists[e][a]: 64-bit keys of what query a of entry entries[e] attends to."""
    if rows is None:
        # every place of the source as one table
        table = torch.cat([src.tail[0].view(-1, src.R), src.pool[0].view(-1, src.R),
                           src.hot[0].view(-1, src.R)])
        table = ref.unpack(table, src.fmt, src.d_v, src.d_rope)
        at_pool = src.n_req * src.T
        at_hot = at_pool + src.pages * src.P
    lists = []
    for i in entries:
        c = stride if count is None else max(0, min(stride, count[i]))
        w = None if words is None else words[i]
        if rows is not None:
            keys = ref.unpack(rows[i], src.fmt, src.d_v, src.d_rope)
        else:
            place, idx = w >> 30, w & 0x3FFFFFFF
            at = np.where(place == 0, i * src.T + idx,
                          np.where(place == 1, at_pool + idx, at_hot + i * src.B + (idx & 0x1FFFFFFF)))
            keys = table[torch.from_numpy(np.where(w == 0xFFFFFFFF, 0, at))]
        per = []
        for a in range(nq):
            js = np.arange(c) if map_ is None else map_[i, a].cpu().numpy()
            js = js[(js >= 0) & (js < c)]
            if w is not None:
                js = js[w[js] != 0xFFFFFFFF]
            per.append(keys[js])
        lists.append(per)
    return lists


def queries(rng, n, nq, heads, width, typ):
    return torch.from_numpy(rng.standard_normal((n, nq, heads, width))).to(typ).cuda()


@pytest.mark.parametrize("fmt,d_v,d_rope", FORMATS)
@pytest.mark.parametrize("tiles", sorted(ROWS))
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_tiles_by_location(fmt, d_v, d_rope, tiles, shape):
    n, nq, heads, mapped = SHAPES[shape]
    k = ROWS[tiles]
    stride = k + k // 3 if mapped else k
    src = Source(100 + tiles, n, fmt, d_v, d_rope)
    rng = src.rng
    words = src.words(n, stride, None, 0.05)
    count = counts(n, stride)
    map_ = None
    if mapped:  # repeats, and entries outside the union
        map_ = torch.from_numpy(rng.integers(-1, stride + 2, (n, nq, k)).astype(np.int32)).cuda()
    q = queries(rng, n, nq, heads, d_v + d_rope, ref.TYPE[fmt])
    scale = (d_v / 4 + 64) ** -0.5
    out, lse, status = attend(src, n, nq, heads, stride, q, scale, words=words, count=count, map_=map_)
    pick = some(n)
    lists = keys_by_query(src, pick, nq, stride, words=words, count=count, map_=map_)
    check(src, q[pick], out[pick], lse[pick], lists, scale)
    assert (status == 0).all()
    again = attend(src, n, nq, heads, stride, q, scale, words=words, count=count, map_=map_)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fmt,d_v,d_rope", FORMATS[:4])
@pytest.mark.parametrize("tiles", [4, 7])
@pytest.mark.parametrize("shape", sorted(SHAPES))
@pytest.mark.parametrize("with_loc", [True, False])
def test_tiles_of_gathered_rows(fmt, d_v, d_rope, tiles, shape, with_loc):
    n, nq, heads, mapped = SHAPES[shape]
    k = ROWS[tiles]
    stride = k + 5 if mapped else k
    src = Source(200 + tiles, n, fmt, d_v, d_rope)
    rng = src.rng
    rows = random_rows(rng, n * stride, fmt, d_v, d_rope).cuda().view(n, stride, src.R)
    words = src.words(n, stride, None, 0.2) if with_loc else None
    count = counts(n, stride)
    map_ = None
    if mapped:
        map_ = torch.from_numpy(rng.integers(-1, stride + 2, (n, nq, k)).astype(np.int32)).cuda()
    q = queries(rng, n, nq, heads, d_v + d_rope, ref.TYPE[fmt])
    scale = (d_v / 4 + 64) ** -0.5
    out, lse, _ = attend(src, n, nq, heads, stride, q, scale, words=words, rows=rows, count=count,
                         map_=map_)
    pick = some(n)
    lists = keys_by_query(src, pick, nq, stride, words=words, rows=rows, count=count, map_=map_)
    check(src, q[pick], out[pick], lse[pick], lists, scale)


@pytest.mark.parametrize("fmt,d_v,d_rope", FORMATS[:4])
@pytest.mark.parametrize("shares", [2, 3, 5])
def test_shares_of_many_tiles(fmt, d_v, d_rope, shares):
    """Two to five shares of several tiles each (by 256 workgroups a call: 100,
    80 and 48 blocks), the last one shorter."""
    n, nq, heads = {2: (25, 1, 127), 3: (20, 1, 128), 5: (12, 2, 60)}[shares]
    stride = 64 * (6 * shares - 2) + 3
    src = Source(300 + shares, n, fmt, d_v, d_rope)
    words = src.words(n, stride, None, 0.05)
    count = counts(n, stride)
    q = queries(src.rng, n, nq, heads, d_v + d_rope, ref.TYPE[fmt])
    out, lse, _ = attend(src, n, nq, heads, stride, q, 0.07, words=words, count=count, shares=True)
    check(src, q, out, lse, keys_by_query(src, range(n), nq, stride, words=words, count=count), 0.07)


def set_rope(rows, fmt, values):
    """rows uint8 [count][R] with their rope parts' first value replaced."""
    typ = ref.TYPE[fmt]
    rows = rows.clone()
    at = rows.shape[1] - 128
    rows[:, at:at + 2] = values.to(typ).view(-1, 1).view(torch.uint8)
    return rows


# log2 of what each tile's scores rise over the first tile's: all of its rows
# (True) or one of them, whose weight the many rows before it then outweigh
RAMPS = {
    "rise": ([9.5 * t for t in range(16)], True),
    "fall": ([-9.5 * t for t in range(16)], True),
    "steps": ([0, 0, 9, 9, 9, 30, 0, -20, 39, 39, 47.5, 0, 0, 60, 61, 0], True),
    "one row late": ([0] * 13 + [9] + [0] * 2, False),
    "rows apart": ([0] * 5 + [8.5] + [0] * 5 + [17.5] + [0] * 3 + [26.5], False),
}


@pytest.mark.parametrize("fmt,d_v,d_rope", [("bf16", 512, 64), ("fp8", 512, 64), ("f16", 512, 64),
                                            ("f16", 256, 64)])
@pytest.mark.parametrize("ramp", sorted(RAMPS))
@pytest.mark.parametrize("shape", ["16", "32"])
def test_reference_grows_in_late_tiles(fmt, d_v, d_rope, ramp, shape):
    """Scores that exceed the first tile's by more than 2^8 in later tiles of one
    workgroup, for some of the query rows of a block (each row sees the ramp
    times its own factor)."""
    n, nq, heads, _ = SHAPES[shape]
    rise, whole = RAMPS[ramp]
    stride = 64 * len(rise) - 11
    src = Source(400, n, fmt, d_v, d_rope)
    rng = src.rng
    step = np.repeat(rise, 64)[:stride].astype(np.float64)
    if not whole:  # one row of the tile
        keep = np.zeros(stride, bool)
        keep[np.arange(len(rise)) * 64 + rng.integers(0, 50, len(rise))] = True
        step = step * keep
    scale = 0.11
    rope = torch.from_numpy(step / (scale * np.log2(np.e)))
    rows = torch.stack([set_rope(random_rows(rng, stride, fmt, d_v, d_rope), fmt, rope)
                        for _ in range(min(n, 3))])
    rows = rows[torch.arange(n) % rows.shape[0]].contiguous().cuda()
    q = queries(rng, n, nq, heads, d_v + d_rope, ref.TYPE[fmt]) * 0.3
    factor = torch.tensor([1.0, 0.0, -1.0, 1.0, 0.5], device="cuda")
    q[..., d_v] = factor[torch.arange(heads, device="cuda") % 5].to(q.dtype)
    q = q.to(ref.TYPE[fmt])
    out, lse, _ = attend(src, n, nq, heads, stride, q, scale, rows=rows)
    pick = some(n)
    check(src, q[pick], out[pick], lse[pick], keys_by_query(src, pick, nq, stride, rows=rows), scale)


@pytest.mark.parametrize("fmt,d_v", [("bf16", 512), ("fp8", 512), ("f16", 256)])
@pytest.mark.parametrize("shape", ["16", "32"])
def test_infinite_scores_and_nan_in_late_tiles(fmt, d_v, shape):
    """In tile 6 of 8: a row of entry 0 whose score is -infinity for some heads
    counts nothing there (and makes the heads NaN whose score is +infinity or
    0 times infinity); a NaN in a row of entry 1 shows in all its heads."""
    n, nq, heads, _ = SHAPES[shape]
    stride = 500
    src = Source(500, n, fmt, d_v, 64)
    rng = src.rng
    rows = random_rows(rng, n * stride, fmt, d_v, 64).view(n, stride, src.R)
    inf = torch.zeros(stride, dtype=torch.float64)
    inf[400] = -np.inf
    rows[0] = set_rope(rows[0], fmt, inf)
    rows[1, 401] = 0xFF  # NaN in every format
    rows = rows.cuda()
    q = queries(rng, n, nq, heads, d_v + 64, ref.TYPE[fmt])
    sign = torch.tensor([1.0, 1.0, -1.0, 0.0, 1.0], device="cuda")[torch.arange(heads) % 5]
    q[..., d_v] = sign.to(q.dtype)
    out, lse, _ = attend(src, n, nq, heads, stride, q, 0.07, rows=rows)
    assert out[1].isnan().all() and lse[1].isnan().all()
    assert out[0][:, sign <= 0].isnan().all() and lse[0][:, sign <= 0].isnan().all()
    pick = [i for i in some(n) if i != 1]
    lists = keys_by_query(src, pick, nq, stride, rows=rows)
    ok = (sign > 0).cpu()
    without = np.r_[0:400, 401:stride]
    check(src, q[:1, :, ok], out[:1, :, ok], lse[:1, :, ok],
          [[keys[without] for keys in lists[0]]], 0.07)
    check(src, q[pick[1:]], out[pick[1:]], lse[pick[1:]], lists[1:], 0.07)


def test_many_rows_of_small_weight():
    """2^18 fp16 rows a workgroup, each with a probability far below fp16's
    normal range, which together weigh up to half: two kinds of rows, so the
    result is their weighted mean in closed form.

    Tolerances, of values of size 1.5 at most: 2^-11 for the probabilities and
    2^-11 for the result, and sums of 2^18 terms, 64 of them at a time for l and
    32 in one product for the values: at most 2^13 additions of 2^-24 each."""
    d_v, heads, nq, stride = 256, 4096, 2, 1 << 18
    src = Source(600, 1, "f16", d_v, 64, B=2)
    one = torch.zeros(2, d_v + 64, dtype=torch.float64)
    one[0, :d_v] = torch.linspace(1.0, 1.5, d_v)
    one[1, :d_v] = -torch.linspace(1.5, 0.75, d_v)
    one[0, d_v] = 16.0
    src.hot[0].copy_(one.half().view(torch.uint8).view(1, 2, src.R))
    keys = ref.unpack(src.hot[0][0], "f16", d_v, 64)
    words = np.full((1, stride), (2 << 30) | 1, np.int64)
    words[0, 77] = 2 << 30
    # scores of the first row over the others': log2 18 to 27
    q = torch.zeros(1, nq, heads, d_v + 64, device="cuda")
    q[..., d_v] = torch.linspace(18.0, 27.0, nq * heads, device="cuda").view(nq, heads)
    q = q.half()
    scale = float(np.log(2.0) / 16)
    out, lse, _ = attend(src, 1, nq, heads, stride, q, scale, words=words)
    s = (q[0].cpu().double() @ keys.T) * np.float64(np.float32(scale))
    w = torch.exp(s[..., 1] - s[..., 0]) * (stride - 1)
    want = (keys[0, :d_v] + w[..., None] * keys[1, :d_v]) / (1 + w[..., None])
    size = 1.5
    tol = (2 * HALF["f16"] + 2 * 2 ** 13 * EPS32) * size
    err = (out[0].cpu().double() - want).abs()
    assert float(err.max()) <= tol, float(err.max() / tol)
    want_lse = s[..., 0] + torch.log1p(w)
    assert ((lse[0].cpu().double() - want_lse).abs() <= (2 ** 13 + 64) * EPS32 * (1 + want_lse)).all()
