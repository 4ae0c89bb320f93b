"""Attention over resolved rows against a plain 64-bit form.

Tolerances.  Let eps32 = 2^-24, h = half a step of the 16-bit type (2^-8 for
bf16, 2^-11 for fp16, relative).  Products of the 16-bit (or e4m3) values are
exact in 32 bits, a score is a sum of at most 576 of them (rounded at most 576
times, plus 8 roundings by scales and the softmax scale): its error is at most
584 eps32 * A with A = scale * max_j sum_d |q_d k_jd|.  So
  |lse - exact| <= 584 eps32 A + (rows + 16) eps32 + 16 eps32 (1 + |lse|)
(the sum of probabilities, its logarithm and its rounding; exp2 and log2 of the
hardware are off by at most a few 32-bit steps).  Each probability carries the
relative error d = 2 * 584 eps32 A + 32 eps32 and is rounded to 16 bits once
(h; fp8 rows: after it was multiplied by the row's scale, one more eps32), then
summed (rows eps32): the output is off by at most (h + d + 2 rows eps32) * S with
S = sum_j p_j |v_j|, and by its own rounding h |out| (a bf16 value below the
smallest normal is not met; fp16's smallest step is 2^-24, half of it 2^-25,
and a probability below fp16's normal range is off by up to 2^-25 of the largest,
which the sum sees rows times at most: rows 2^-25 max|v|).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import attend_reference as ref

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "fp8": 2.0 ** -8}


class Source:
    """A context of random rows in every place, without the resolver's state."""

    def __init__(self, seed, n_req, fmt, d_v, d_rope, *, T=19, P=8, pages=21, B=70, H=64,
                 n_layers=1, poison=True):
        from hierarchical_sparse_kv_resolve_amd import Context
        rng = np.random.default_rng(seed)
        self.rng, self.fmt, self.d_v, self.d_rope = rng, fmt, d_v, d_rope
        self.n_req, self.T, self.P, self.pages, self.B = n_req, T, P, pages, B
        self.R = ref.row_bytes(fmt, d_v, d_rope)
        self.ctx = Context(n_req=n_req, n_layers=n_layers, history_rows=H, max_new_rows=0,
                           page_rows=P, tail_rows=T, hot_slots=B, row_bytes=self.R, sel_cap=B,
                           pool_pages=pages)
        make = lambda c: ref.random_rows(rng, c, fmt, d_v, d_rope).cuda()  # noqa: E731
        self.tail = [make(n_req * T).view(n_req, T, self.R) for _ in range(n_layers)]
        self.pool = [make(pages * P).view(pages, P, self.R) for _ in range(n_layers)]
        self.hot = [make(n_req * B).view(n_req, B, self.R) for _ in range(n_layers)]
        self.host = [torch.empty(n_req, H, self.R, dtype=torch.uint8, pin_memory=True)
                     for _ in range(n_layers)]
        for l in range(n_layers):
            self.ctx.bind_layer(l, self.tail[l], self.pool[l], self.hot[l], self.host[l])

    def words(self, n, stride, req, invalid=0.0):
        """Random location words int64 [n][stride] of every place."""
        rng = self.rng
        place = rng.integers(0, 3, (n, stride))
        index = np.where(place == 0, rng.integers(0, self.T, (n, stride)),
                         np.where(place == 1, rng.integers(0, self.pages * self.P, (n, stride)),
                                  rng.integers(0, self.B, (n, stride))))
        fresh = (rng.random((n, stride)) < 0.3) & (place == 2)
        w = (place << 30) | index | (fresh.astype(np.int64) << 29)
        return np.where(rng.random((n, stride)) < invalid, 0xFFFFFFFF, w)

    def row_of(self, layer, r, word):
        place, idx = word >> 30, word & 0x3FFFFFFF
        if place == 0:
            return self.tail[layer][r, idx]
        if place == 1:
            return self.pool[layer].view(-1, self.R)[idx]
        return self.hot[layer][r, idx & 0x1FFFFFFF]


def to_dev(words):
    return torch.from_numpy(words.astype(np.uint32).view(np.int32)).cuda()


def check(src, q, out, lse, lists, scale):
    """out and lse against the plain form; lists[i][a] = keys float64 of query a."""
    n, nq, heads, _ = q.shape
    h = HALF[src.fmt]
    q, out, lse = q.cpu(), out.cpu().double(), lse.cpu().double()
    for i in range(n):
        for a in range(nq):
            keys = lists[i][a]
            rows = keys.shape[0]
            o, s, spread = ref.attend(q[i, a], keys, src.d_v, scale)
            if rows == 0:
                assert (out[i, a] == 0).all() and (lse[i, a] == -np.inf).all(), (i, a)
                continue
            size = ref.score_size(q[i, a], keys, scale)
            d = 584 * EPS32 * size
            tol_lse = d + (rows + 16) * EPS32 + 16 * EPS32 * (1 + s.abs())
            err = (lse[i, a] - s).abs()
            assert (err <= tol_lse).all(), (i, a, float((err / tol_lse).max()))
            tol = (h + 2 * d + 32 * EPS32 + 2 * rows * EPS32)[:, None] * spread + h * o.abs()
            if src.fmt == "f16":
                tol = tol + 2.0 ** -25 * (1 + rows * keys[:, :src.d_v].abs().max())
            err = (out[i, a] - o).abs()
            assert (err <= tol).all(), (i, a, float((err / tol).max()))


def run(src, n, nq, heads, stride, *, count=None, invalid=0.0, map_k=0, rows=False, req=None,
        scale=None, q=None, layer=0, loc_with_rows=True, words=None, workspace=True):
    from hierarchical_sparse_kv_resolve_amd import Context
    rng, D = src.rng, src.d_v + src.d_rope
    typ = ref.TYPE[src.fmt]
    scale = scale if scale is not None else (src.d_v / 4 + 64) ** -0.5
    if words is None:
        words = src.words(n, stride, req, invalid)
    loc = to_dev(words)
    if q is None:
        q = torch.from_numpy(rng.standard_normal((n, nq, heads, D))).to(typ).cuda()
    out = torch.full((n, nq, heads, src.d_v), 7.0, dtype=typ, device="cuda")
    lse = torch.full((n, nq, heads), 7.0, dtype=torch.float32, device="cuda")
    map_ = None
    if map_k:
        # some indices out of range, some repeated
        map_ = torch.from_numpy(rng.integers(-1, stride + 2, (n, nq, map_k)).astype(np.int32)).cuda()
    gathered = None
    if rows:
        gathered = ref.random_rows(rng, n * stride, src.fmt, src.d_v, src.d_rope).cuda()
        gathered = gathered.view(n, stride, src.R)
    cnt = None if count is None else torch.tensor(count, dtype=torch.int32, device="cuda")
    rid = None if req is None else torch.tensor(req, dtype=torch.int32, device="cuda")
    status = torch.zeros(n, dtype=torch.int32, device="cuda")
    need = Context.attend_workspace(n, nq, heads, src.d_v, map_k or stride)
    ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda") if workspace else None
    src.ctx.attend_rows(layer, n, rid, q, out, fmt=src.fmt, d_v=src.d_v, d_rope=src.d_rope,
                        scale=scale, stride=stride, loc=loc if loc_with_rows or not rows else None,
                        rows=gathered, count=cnt, map_=map_, lse=lse, status=status, workspace=ws)
    torch.cuda.synchronize()
    if ws is not None:
        assert (ws[need:] == 0x7F).all(), "the workspace's end was written past"
    lists = []
    for i in range(n):
        r = i if req is None else req[i]
        c = stride if count is None else max(0, min(stride, count[i]))
        if not 0 <= r < src.n_req:
            c = 0
        keys = []
        if c:
            if rows:
                raw = gathered[i]
            else:
                raw = torch.stack([src.row_of(layer, r, int(w)) if w != 0xFFFFFFFF else src.hot[0][0, 0]
                                   for w in words[i]])
            keys = ref.unpack(raw, src.fmt, src.d_v, src.d_rope)
        per = []
        for a in range(nq):
            js = np.arange(c) if map_ is None else map_[i, a].cpu().numpy()
            js = js[(js >= 0) & (js < c)]
            if not rows or loc_with_rows:
                js = js[words[i][js] != 0xFFFFFFFF] if len(js) else js
            per.append(keys[js] if c else torch.zeros(0, src.d_v + src.d_rope, dtype=torch.float64))
        lists.append(per)
    return q, out, lse, lists, scale, status


FORMATS = [("bf16", 512, 64), ("fp8", 512, 64), ("f16", 512, 64), ("bf16", 256, 64),
           ("fp8", 256, 0), ("f16", 256, 0), ("fp8", 512, 0), ("fp8", 256, 64)]


@pytest.mark.parametrize("fmt,d_v,d_rope", FORMATS)
@pytest.mark.parametrize("heads,stride", [(1, 1), (16, 64), (23, 65), (5, 130), (64, 63), (128, 33)])
def test_locations(fmt, d_v, d_rope, heads, stride):
    src = Source(1, 2, fmt, d_v, d_rope)
    check(src, *run(src, 2, 1, heads, stride)[:5])


@pytest.mark.parametrize("fmt,d_v,d_rope", FORMATS[:3])
@pytest.mark.parametrize("n,nq,heads", [(1, 1, 16), (3, 4, 16), (2, 3, 7), (1, 2, 40), (5, 1, 100)])
def test_long_selections_ragged_counts(fmt, d_v, d_rope, n, nq, heads):
    """Counts of none, one, all, below 0 and above the stride; left-out words."""
    src = Source(2, 5, fmt, d_v, d_rope)
    count = [1500, 0, 1, 777, -3][:n]
    got = run(src, n, nq, heads, 1301, count=count, invalid=0.1)
    check(src, *got[:5])
    assert (got[5] == 0).all()


@pytest.mark.parametrize("fmt,d_v,d_rope", FORMATS[:3])
@pytest.mark.parametrize("nq,heads,k", [(4, 16, 200), (2, 70, 64), (3, 1, 1), (2, 33, 500)])
def test_verify_block_map(fmt, d_v, d_rope, nq, heads, k):
    """Each query its own entries of the union, with indices out of range."""
    src = Source(3, 3, fmt, d_v, d_rope)
    check(src, *run(src, 3, nq, heads, 310, count=[310, 0, 100], invalid=0.05, map_k=k)[:5])


@pytest.mark.parametrize("fmt,d_v,d_rope", FORMATS[:4])
@pytest.mark.parametrize("with_loc", [True, False])
def test_gathered_rows(fmt, d_v, d_rope, with_loc):
    src = Source(4, 3, fmt, d_v, d_rope)
    check(src, *run(src, 3, 2, 16, 150, count=[150, 3, 0], invalid=0.2, rows=True,
                    loc_with_rows=with_loc)[:5])


def test_request_ids_and_bad_ones():
    """Entries name requests in any order, one twice; ids out of range get
    nothing and KVR_E_ARG."""
    src = Source(5, 6, "bf16", 512, 64)
    got = run(src, 6, 1, 16, 90, req=[4, 0, 6, 2, -1, 4])
    check(src, *got[:5])
    assert got[5].cpu().tolist() == [0, 0, -1, 0, -1, 0]


def test_second_layer():
    src = Source(6, 2, "fp8", 512, 64, n_layers=3)
    check(src, *run(src, 2, 1, 16, 90, layer=2)[:5])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "f16"])
def test_locations_outside_their_place(fmt):
    """Words outside their place are left out and reported, the others count."""
    src = Source(7, 3, fmt, 512, 64)
    words = src.words(3, 80, None)
    words[0, 7] = src.T                              # past the tail
    words[0, 70] = (1 << 30) | (src.pages * src.P)   # past the pool
    words[2, 79] = (2 << 30) | src.B                 # past the hot cache
    words[2, 0] = (3 << 30) | 5                      # no place
    q, out, lse, lists, scale, status = _run_bad(src, words)
    check(src, q, out, lse, lists, scale)
    assert status.cpu().tolist() == [-2, 0, -2]


def _run_bad(src, words):
    """A call with words outside their places: the plain form leaves them out."""
    n, stride = words.shape
    typ = ref.TYPE[src.fmt]
    q = torch.from_numpy(src.rng.standard_normal((n, 1, 20, src.d_v + src.d_rope))).to(typ).cuda()
    out = torch.zeros(n, 1, 20, src.d_v, dtype=typ, device="cuda")
    lse = torch.zeros(n, 1, 20, device="cuda")
    status = torch.zeros(n, dtype=torch.int32, device="cuda")
    ws = torch.zeros(src.ctx.attend_workspace(n, 1, 20, src.d_v, stride), dtype=torch.uint8,
                     device="cuda")
    src.ctx.attend_rows(0, n, None, q, out, fmt=src.fmt, d_v=src.d_v, d_rope=src.d_rope, scale=0.1,
                        stride=stride, loc=to_dev(words), lse=lse, status=status, workspace=ws)
    limit = {0: src.T, 1: src.pages * src.P, 2: src.B, 3: 0}
    lists = []
    for i in range(n):
        good = [int(w) for w in words[i]
                if (w & (0x1FFFFFFF if w >> 30 == 2 else 0x3FFFFFFF)) < limit[int(w >> 30)]]
        lists.append([ref.unpack(torch.stack([src.row_of(0, i, w) for w in good]), src.fmt, src.d_v,
                                 src.d_rope)])
    return q, out, lse, lists, 0.1, status


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "f16"])
def test_rows_left_out_may_hold_anything(fmt):
    """NaN and infinities in rows past the count, in rows of left-out words and
    in places no word names do not show; one in a row that takes part does."""
    src = Source(8, 2, fmt, 512, 64)
    bad = torch.full((src.R,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every format
    typ = ref.TYPE[fmt]
    n, stride, heads = 2, 100, 16
    rows = ref.random_rows(src.rng, n * stride, fmt, 512, 64).cuda().view(n, stride, -1)
    words = np.zeros((n, stride), dtype=np.int64)
    words[0, 10:20] = 0xFFFFFFFF
    rows[0, 10:20] = bad
    rows[1, 33:] = bad
    count = torch.tensor([100, 33], dtype=torch.int32, device="cuda")
    q = torch.from_numpy(src.rng.standard_normal((n, 1, heads, 576))).to(typ).cuda()
    out = torch.empty(n, 1, heads, 512, dtype=typ, device="cuda")
    lse = torch.empty(n, 1, heads, device="cuda")
    ws = torch.full((src.ctx.attend_workspace(n, 1, heads, 512, stride),), 0xFF,
                    dtype=torch.uint8, device="cuda")

    def call():
        src.ctx.attend_rows(0, n, None, q, out, fmt=fmt, d_v=512, d_rope=64, scale=0.07,
                            stride=stride, loc=to_dev(words), rows=rows, count=count, lse=lse,
                            workspace=ws)
        torch.cuda.synchronize()

    call()
    keys = [ref.unpack(rows[i], fmt, 512, 64) for i in range(n)]
    pick = np.r_[0:10, 20:100]
    check(src, q, out, lse, [[keys[0][pick]], [keys[1][:33]]], 0.07)
    rows[0, 50] = bad
    call()
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert not out[1].isnan().any() and not lse[1].isnan().any()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "f16"])
def test_scores_far_apart(fmt):
    """Scores over +-600: every head's weight sits on few rows, the running
    maximum grows in late tiles, and exponentials underflow."""
    src = Source(9, 1, fmt, 512, 64, B=600)
    words = ((2 << 30) | np.arange(600)[None]).astype(np.int64)
    ramp = np.linspace(0.01, 6.0, 600)
    rows = ref.random_rows(src.rng, 600, fmt, 512, 64)
    x = ref.unpack(rows, fmt, 512, 64) * torch.from_numpy(ramp)[:, None]
    if fmt == "fp8":
        groups = rows[:, 512:528].contiguous().view(torch.float32) * torch.from_numpy(ramp)[:, None].float()
        rows[:, 512:528] = groups.contiguous().view(torch.uint8)
        rows[:, 528:] = x[:, 512:].to(torch.bfloat16).contiguous().view(torch.uint8)
    else:
        rows = x.to(ref.TYPE[fmt]).view(torch.uint8)
    src.hot[0][0] = rows.cuda()
    check(src, *run(src, 1, 2, 16, 600, words=words, scale=0.9)[:5])
    check(src, *run(src, 1, 2, 16, 600, words=words, scale=-0.9)[:5])
    check(src, *run(src, 1, 1, 16, 600, words=words, scale=0.0)[:5])


@pytest.mark.parametrize("stride", [5, 70, 700])
def test_infinite_scores(stride):
    """A head whose scores are all -infinity is as one without rows, one with
    +infinity is NaN, and neither touches its neighbours."""
    src = Source(18, 2, "bf16", 512, 64)
    q = torch.zeros(2, 1, 20, 576, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 3, 0] = -float("inf")
    q[1, 0, 18, 1] = float("inf")
    rows = torch.ones(2, stride, 576, dtype=torch.bfloat16, device="cuda").view(torch.uint8)
    out = torch.full((2, 1, 20, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 1, 20), 7.0, device="cuda")
    ws = torch.empty(src.ctx.attend_workspace(2, 1, 20, 512, stride), dtype=torch.uint8, device="cuda")
    src.ctx.attend_rows(0, 2, None, q, out, fmt="bf16", d_v=512, d_rope=64, scale=0.5,
                        stride=stride, rows=rows, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert (out[0, 0, 3] == 0).all() and lse[0, 0, 3].item() == -np.inf
    assert out[1, 0, 18].isnan().all() and lse[1, 0, 18].isnan()
    keep = torch.ones(2, 1, 20, dtype=torch.bool, device="cuda")
    keep[0, 0, 3] = keep[1, 0, 18] = False
    # p = 1 for every row: out is 1 up to the roundings of 1 / l, lse is ln(stride)
    assert (out[keep] == 1).all()
    assert ((lse[keep] - np.log(stride)).abs() <= 32 * EPS32 * (1 + np.log(stride))).all()


def test_strided_queries():
    """Queries as a slice of a larger tensor (odd head and entry strides)."""
    src = Source(10, 3, "bf16", 512, 64)
    for pad in (8, 1, 3):
        big = torch.from_numpy(src.rng.standard_normal((3, 2, 20, 576 + pad))).bfloat16().cuda()
        q = big[:, :, 1:17, pad:]
        check(src, *run(src, 3, 2, 16, 70, q=q)[:5])
        q = big[:, :1, :16, :576].expand(3, 2, 16, 576)  # one query for both
        check(src, *run(src, 3, 2, 16, 70, q=q)[:5])


def test_empty_calls():
    src = Source(11, 3, "fp8", 512, 64)
    run(src, 0, 1, 16, 50)
    for kw in (dict(stride=0), dict(stride=40, count=[0, 0, 0]), dict(stride=40, invalid=1.1)):
        got = run(src, 3, 2, 16, **kw)
        check(src, *got[:5])


def test_same_result_twice_and_on_another_stream():
    src = Source(12, 4, "bf16", 512, 64)
    words = src.words(4, 1000, None)
    q = torch.randn(4, 1, 16, 576, device="cuda").bfloat16()
    a = run(src, 4, 1, 16, 1000, words=words, q=q)
    b = run(src, 4, 1, 16, 1000, words=words, q=q)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = run(src, 4, 1, 16, 1000, words=words, q=q)
    assert torch.equal(a[1], c[1]) and torch.equal(a[2], c[2])


def test_two_calls_at_once():
    """Calls on two streams with workspaces of their own."""
    src = Source(16, 6, "fp8", 512, 64, n_layers=2)
    n, heads, stride = 6, 20, 900
    loc = [to_dev(src.words(n, stride, None, 0.1)) for _ in range(2)]
    q = [torch.randn(n, 1, heads, 576, device="cuda").bfloat16() for _ in range(2)]
    need = src.ctx.attend_workspace(n, 1, heads, 512, stride)
    outs = [[torch.zeros(n, 1, heads, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            for _ in range(2)]
    ws = [torch.zeros(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()

    def call(i, out, stream=None):
        src.ctx.attend_rows(i, n, None, q[i], out, fmt="fp8", d_v=512, d_rope=64, scale=0.07,
                            stride=stride, loc=loc[i], workspace=ws[i], stream=stream)

    for i in range(2):
        call(i, outs[0][i])
        torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            call(i, outs[1][i], streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[0][i], outs[1][i])
        assert not torch.equal(outs[0][0], outs[0][1])


def test_every_share_count():
    """Selections of one to many tiles, so that every number of shares occurs,
    with counts that leave the last shares empty."""
    src = Source(17, 3, "bf16", 512, 64, B=2000)
    for stride in (64, 65, 128, 300, 640, 1999):
        for count in (None, [stride, 64, 1]):
            check(src, *run(src, 3, 1, 16, stride, count=count)[:5])


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("n,nq,heads,stride", [(1, 16, 100, 70), (3, 40, 33, 130), (9, 2, 17, 64)])
def test_many_query_rows(fmt, n, nq, heads, stride):
    """Few selections shared by many blocks of query rows, in numbers that are
    no multiples of one another."""
    check(Source(19, n, fmt, 512, 64), *run(Source(19, n, fmt, 512, 64), n, nq, heads, stride)[:5])


def test_captured_and_replayed():
    """One captured call, replayed with new contents and eager work between."""
    src = Source(13, 3, "fp8", 512, 64)
    n, heads, stride = 3, 16, 700
    loc = to_dev(src.words(n, stride, None))
    q = torch.randn(n, 1, heads, 576, device="cuda").bfloat16()
    out = torch.zeros(n, 1, heads, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(n, 1, heads, device="cuda")
    ws = torch.zeros(src.ctx.attend_workspace(n, 1, heads, 512, stride), dtype=torch.uint8,
                     device="cuda")
    ws2 = torch.zeros_like(ws)

    def call(o, l, w):
        src.ctx.attend_rows(0, n, None, q, o, fmt="fp8", d_v=512, d_rope=64, scale=0.07,
                            stride=stride, loc=loc, lse=l, workspace=w)

    call(out, lse, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out, lse, ws)
    for _ in range(4):
        q.copy_(torch.randn(n, 1, heads, 576, device="cuda"))
        loc.copy_(to_dev(src.words(n, stride, None, 0.1)))
        out.zero_()
        o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
        g.replay()
        call(o2, l2, ws2)
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_pool_offsets_past_32_bits():
    """Rows behind the first 4 GiB of a pool are read at their own place."""
    R = 1152
    pages = (5 << 30) // (64 * R)
    from hierarchical_sparse_kv_resolve_amd import Context
    ctx = Context(n_req=1, n_layers=1, history_rows=64, max_new_rows=0, page_rows=64, tail_rows=0,
                  hot_slots=1, row_bytes=R, sel_cap=64, pool_pages=pages)
    pool = torch.zeros(pages, 64, R, dtype=torch.uint8, device="cuda")
    host = torch.empty(1, 64, R, dtype=torch.uint8, pin_memory=True)
    hot = torch.zeros(1, 1, R, dtype=torch.uint8, device="cuda")
    ctx.bind_layer(0, None, pool, hot, host)
    rng = np.random.default_rng(14)
    idx = np.sort(rng.choice(np.arange(pages * 64 - 100000, pages * 64), 200, replace=False))
    rows = ref.random_rows(rng, 200, "bf16", 512, 64)
    pool.view(-1, R)[torch.from_numpy(idx).cuda()] = rows.cuda()
    src = type("S", (), dict(fmt="bf16", d_v=512))
    q = torch.randn(1, 1, 16, 576, device="cuda").bfloat16()
    out = torch.zeros(1, 1, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(1, 1, 16, device="cuda")
    ws = torch.zeros(ctx.attend_workspace(1, 1, 16, 512, 200), dtype=torch.uint8, device="cuda")
    ctx.attend_rows(0, 1, None, q, out, fmt="bf16", d_v=512, d_rope=64, scale=0.07, stride=200,
                    loc=to_dev((1 << 30) | idx[None].astype(np.int64)), lse=lse, workspace=ws)
    check(src, q, out, lse, [[ref.unpack(rows, "bf16", 512, 64)]], 0.07)


def test_refusals():
    from hierarchical_sparse_kv_resolve_amd import KvrError
    src = Source(15, 2, "bf16", 512, 64)
    q = torch.zeros(2, 1, 16, 576, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(2, 1, 16, 512, dtype=torch.bfloat16, device="cuda")
    loc = torch.zeros(2, 40, dtype=torch.int32, device="cuda")
    ws = torch.zeros(src.ctx.attend_workspace(2, 1, 16, 512, 40) + 16, dtype=torch.uint8,
                     device="cuda")
    good = dict(layer=0, n=2, req_ids=None, q=q, out=out, fmt="bf16", d_v=512, d_rope=64, scale=0.1,
                stride=40, loc=loc, workspace=ws)
    src.ctx.attend_rows(**good)

    def refused(error, match, **kw):
        with pytest.raises(error, match=match):
            src.ctx.attend_rows(**{**good, **kw})

    refused(ValueError, "unknown row format", fmt="int8")
    refused(TypeError, "q: expected float16", fmt="f16")
    refused(TypeError, "q: expected a GPU tensor", q=q.cpu())
    refused(ValueError, "q: shape", q=q[:1])
    refused(ValueError, "dimensions", q=q[0])
    refused(ValueError, "last dimension", q=torch.zeros(2, 1, 576, 16, dtype=torch.bfloat16,
                                                        device="cuda").transpose(2, 3))
    refused(TypeError, "out: expected bfloat16", out=out.float())
    refused(ValueError, "out: the tensor is not contiguous",
            out=torch.zeros(2, 1, 16, 513, dtype=torch.bfloat16, device="cuda")[..., :512])
    refused(ValueError, "lse: shape", lse=torch.zeros(2, 16, device="cuda"))
    refused(TypeError, "map: expected int32", map_=torch.zeros(2, 1, 4, device="cuda"))
    refused(TypeError, "count: expected int32", count=torch.zeros(2, device="cuda"))
    refused(TypeError, "loc: expected int32", loc=loc.long())
    refused(TypeError, "status: expected int32", status=torch.zeros(2, device="cuda"))
    refused(ValueError, "loc: ", loc=loc[:, :39].contiguous())
    refused(ValueError, "count: ", count=torch.zeros(1, dtype=torch.int32, device="cuda"))
    refused(KvrError, "layer 1 outside", layer=1)
    refused(KvrError, "rows or loc", loc=None)
    refused(KvrError, "have 656 bytes", fmt="fp8")
    refused(KvrError, "negative stride", stride=-1)
    with pytest.raises(KvrError, match="d_v 512 with d_rope 32"):
        src.ctx.attend_rows(**{**good, "d_rope": 32, "q": q[..., :544]})
    with pytest.raises(KvrError, match="request count"):
        src.ctx.attend_rows(**{**good, "n": 3, "q": torch.cat([q, q[:1]]),
                               "out": torch.cat([out, out[:1]]), "loc": torch.cat([loc, loc[:1]])})
    assert out.isfinite().all()


@pytest.mark.parametrize("part", ["tail", "pool", "hot"])
def test_layer_buffers_off_16_bytes_are_refused(part):
    """A layer bound 8 bytes off is refused before anything is launched; gathered
    rows do not read it."""
    from hierarchical_sparse_kv_resolve_amd import KvrError
    src = Source(20, 2, "bf16", 512, 64)
    bufs = {k: getattr(src, k)[0] for k in ("tail", "pool", "hot")}
    flat = torch.zeros(bufs[part].numel() + 16, dtype=torch.uint8, device="cuda")
    src.ctx.bind_layer(0, **{**bufs, part: flat[8:-8]}, host=src.host[0])
    q = torch.zeros(2, 1, 16, 576, dtype=torch.bfloat16, device="cuda")
    out = torch.full((2, 1, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    kw = dict(fmt="bf16", d_v=512, d_rope=64, scale=0.1, stride=40)
    with pytest.raises(KvrError, match="not aligned to 16 bytes"):
        src.ctx.attend_rows(0, 2, None, q, out, **kw,
                            loc=torch.zeros(2, 40, dtype=torch.int32, device="cuda"))
    assert (out == 7).all()
    src.ctx.attend_rows(0, 2, None, q, out, **kw,
                        rows=torch.zeros(2, 40, src.R, dtype=torch.uint8, device="cuda"))
    assert (out == 0).all()
