"""The drafter's window in 8 bits: codes and scales bit for bit against the plain
form, the rows read back, lengths, and attention in 64 bits.

Codes.  A scale is a power of two, so x / scale is exact in 32 bits for values of
16 and 32 bits and a code is its nearest e4m3 value: no tolerance.  Rows read back
are code * scale: exact in 32 bits and in bf16 (3 mantissa bits), rounded once in
fp16.

Attention.  eps32 = 2^-24, h = 2^-8 (half a step of bf16, relative).  Queries and
codes are exact in bf16, products exact in 32 bits; a score is a sum of at most
256 of them and two scalings: off by at most c eps32 A, c = 264, A = scale max_j
sum_d |q_d k_jd|.  So |lse - exact| <= c eps32 A + (rows + 16) eps32 + 16 eps32
(1 + |lse|) as in the tests of attention over resolved rows (sum, logarithm,
hardware exp2 and log2); each probability is off by d = 2 c eps32 A + 32 eps32
and rounded once to bf16 (h), their sums by rows eps32, and the output by its own
rounding: |out - exact| <= (h + d + 2 rows eps32) S + h |out|, S = sum p |v|.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import draft_reference as ref

pytestmark = pytest.mark.gpu

EPS32 = 2.0 ** -24
H = 2.0 ** -8
TYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Ring:
    """A ring of the package beside its plain form (layer `layer` of several)."""

    def __init__(self, n_req, W, C, kv, d, layers=1, layer=0):
        from hierarchical_sparse_kv_resolve_amd import DraftRing
        self.ref = ref.Window(n_req, W, C, kv, d)
        self.layer = layer
        # what the ring holds before its first write: NaN codes, scales of any size
        self.codes = torch.full((layers, n_req, C // 64, kv, 2, 64 * d), 0x7F, dtype=torch.uint8,
                                device=DEV)
        self.scales = torch.full((layers, n_req, C // 64, kv, 2), 255, dtype=torch.uint8,
                                 device=DEV)
        self.length = torch.full((n_req,), 99, dtype=torch.int32, device=DEV)
        self.high = torch.full((n_req,), 7, dtype=torch.int32, device=DEV)
        self.ring = DraftRing(n_req, W, C, 0, None, self.length, self.high)
        self.ring.bind_kv(layers, kv, d, self.codes, self.scales)
        self.ring.reset()
        self.written = np.zeros((n_req, C // 64), dtype=bool)

    def write(self, reqs, k, v, count=None, strided=False, typ="f32"):
        """k, v float64 [n, rows, kv, d] (values exact in `typ`)."""
        rows = k.shape[1]
        kt, vt = (torch.from_numpy(x).to(TYPE[typ]).to(DEV) for x in (k, v))
        if strided:  # slices of one projection's output, off any alignment
            both = torch.zeros(*k.shape[:3], 2 * k.shape[3] + 3, dtype=TYPE[typ], device=DEV)
            both[..., 1:1 + k.shape[3]], both[..., 2 + k.shape[3]:-1] = kt, vt
            kt, vt = both[..., 1:1 + k.shape[3]], both[..., 2 + k.shape[3]:-1]
        status = torch.full((len(reqs),), 9, dtype=torch.int32, device=DEV)
        self.ring.write_kv(self.layer, len(reqs), i32(reqs), kt, vt,
                           None if count is None else i32(count), status)
        torch.cuda.synchronize()
        assert (status == 0).all()
        k64, v64 = (torch.from_numpy(x).to(TYPE[typ]).double().numpy() for x in (k, v))
        for i, r in enumerate(reqs):
            m = rows if count is None else count[i]
            self.ref.write(r, k64[i, :m], v64[i, :m])
            a = int(self.ref.length[r])
            for p in range(a, a + m):
                self.written[r, p // 64 % self.written.shape[1]] = True

    def advance(self, reqs, rows, count=None):
        self.ring.advance(len(reqs), i32(reqs), rows, None if count is None else i32(count))
        for i, r in enumerate(reqs):
            self.ref.advance(r, rows if count is None else count[i])

    def rollback(self, reqs, keep):
        status = torch.full((len(reqs),), 9, dtype=torch.int32, device=DEV)
        self.ring.rollback(len(reqs), i32(reqs), i32(keep), status)
        assert (status == 0).all()
        self.ref.length[np.asarray(reqs)] = keep

    def check(self):
        """Every written block bit for bit (a NaN code as any NaN)."""
        codes, scales = self.ref.device_layout()
        got = self.codes[self.layer].cpu().numpy()
        w = self.written
        assert np.array_equal(self.scales[self.layer].cpu().numpy()[w], scales[w])
        a, b = got[w], codes[w]
        same = (a == b) | (((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F))
        assert same.all(), np.argwhere(~same)[:5]
        assert np.array_equal(self.length.cpu().numpy(), self.ref.length)
        assert np.array_equal(self.high.cpu().numpy(), self.ref.high)
        # blocks never written stay as they were
        assert (got[~w] == 0x7F).all()


def values(rng, shape, spread=1.0):
    """Normal values of tokens of different sizes, exact in bf16."""
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[:2] + (1, 1)))
    return torch.from_numpy(x).bfloat16().double().numpy()


@pytest.mark.parametrize("kv,d", [(1, 64), (3, 128), (2, 256)])
@pytest.mark.parametrize("typ", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("strided", [False, True])
def test_write_in_steps(kv, d, typ, strided):
    """Appends of every size into a ring that wraps, rolled back at times."""
    rng = np.random.default_rng(kv * d + strided)
    n, W, C = 3, 100, 256
    R = Ring(n, W, C, kv, d)
    for step in range(24):
        reqs = sorted(rng.choice(n, size=int(rng.integers(1, n + 1)), replace=False).tolist())
        rows = int(rng.choice([1, 1, 2, 5, 63, 64, 65, 130, C - 63]))
        k = np.clip(values(rng, (len(reqs), rows, kv, d)), -6e4, 6e4)
        v = np.clip(values(rng, (len(reqs), rows, kv, d)), -6e4, 6e4)
        count = rng.integers(0, rows + 1, len(reqs)).tolist() if step % 2 else None
        R.write(reqs, k, v, count, strided, typ)
        R.check()
        R.advance(reqs, rows, count)
        if rows <= 5:  # some of the new rows are rejected
            keep = [int(rng.integers(max(0, R.ref.high[r] - (C - W), R.ref.length[r] - rows),
                                     R.ref.length[r] + 1)) for r in reqs]
            R.rollback(reqs, keep)
    R.check()


def test_scales_follow_their_rows():
    """An outlier raises its block's scale and lowers it when it goes: codes of rows
    kept keep their values but for those that fell below the smallest code."""
    rng = np.random.default_rng(5)
    R = Ring(1, 60, 128, 1, 64)
    one = lambda size: values(rng, (1, 1, 1, 64), 0.0) * size  # noqa: E731
    for step, size in enumerate([1.0] * 10 + [2.0 ** 20] + [1.0] * 20 + [2.0 ** -30] * 3 + [0.0]
                                + [1.0] * 150):
        R.write([0], one(size), one(size))
        R.advance([0], 1)
        if step == 10:  # the outlier: small rows of its block have gone to 0
            assert R.ref.exp[0, 0, 0, 0] > 5 and (R.ref.rows(0, 0, 5)[0] == 0).all()
        R.check()
    assert R.ref.exp[0, 0, 0, 0] < -5  # overwritten since


def test_zeros_and_the_ends_of_the_range():
    rng = np.random.default_rng(6)
    R = Ring(2, 64, 192, 1, 64)
    k = np.zeros((2, 70, 1, 64))
    v = np.zeros((2, 70, 1, 64))
    k[1] = 2.0 ** 126 * rng.standard_normal((70, 1, 64)).clip(-1, 1)
    v[1] = 2.0 ** -126 * rng.standard_normal((70, 1, 64)).clip(-1, 1)
    k, v = (torch.from_numpy(x).float().double().numpy() for x in (k, v))
    R.write([0, 1], k, v)
    R.advance([0, 1], 70)
    R.check()
    assert (R.ref.exp[0, :2] == -100).all()
    # the large block becomes one of zeros, the zero block a large one, then again
    for flip in (1, 0, 1):
        R.write([0, 1], k[[flip, 1 - flip]], v[[flip, 1 - flip]])
        R.advance([0, 1], 70)
        R.check()


def test_exact_borders():
    """Values at and beside 448 times a power of two, and ties between codes."""
    base = np.array([448.0, 449.0, 447.0, 464.0, 432.0, 17.0, 19.0, 1.0625, 1.1875, 2.0 ** -9,
                     2.0 ** -10, 1.5 * 2.0 ** -9, 2.0 ** -7 + 2.0 ** -10, 0.0, -448.0, -1.0625])
    for power in (0, -40, 60):
        R = Ring(1, 64, 128, 1, 64)
        x = np.zeros((1, len(base), 1, 64))
        for t in range(len(base)):
            x[0, t, 0, :16] = np.roll(base, t) * 2.0 ** power * (1 if t else 0.5)
        x = torch.from_numpy(x).float().double().numpy()
        for t in range(len(base)):
            R.write([0], x[:, t:t + 1], x[:, t:t + 1][..., ::-1].copy())
            R.advance([0], 1)
            R.check()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("where", ["k", "v"])
def test_values_that_are_not_finite(bad, where):
    rng = np.random.default_rng(8)
    n, kv, d, W, C = 1, 2, 64, 64, 192
    R = Ring(n, W, C, kv, d)
    k, v = values(rng, (n, 100, kv, d)), values(rng, (n, 100, kv, d))
    (k if where == "k" else v)[0, 70, 1, 5] = bad
    R.write([0], k, v)
    R.advance([0], 100)
    R.check()
    R.write([0], k[:, :9], v[:, :9])  # and as rows kept of a touched block
    R.check()
    # queries that see the token get NaN in its head, the others do not
    q = torch.randn(1, 9, 2 * kv, d, device=DEV).bfloat16()
    out, lse = attend(R, [0], q, "causal")
    assert out.isfinite()[:, :, :2].all() and lse.isfinite()[:, :, :2].all()
    assert out.isnan()[:, :, 2:].all() and lse.isnan()[:, :, 2:].all()
    R.advance([0], 9)
    more = values(rng, (1, 40, kv, d))
    R.write([0], more, more)
    q = torch.randn(1, 40, 2 * kv, d, device=DEV).bfloat16()
    out, lse = attend(R, [0], q, "causal")
    # query j sees positions 109 + j - 63 on: past the token from j = 25 on
    assert out.isnan()[:, :25, 2:].all() and out.isfinite()[:, 25:].all()
    assert lse.isfinite()[:, 25:].all()


@pytest.mark.parametrize("typ", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kv,d,W,C", [(2, 64, 100, 128), (1, 128, 64, 64), (3, 256, 130, 256)])
def test_read_back(typ, kv, d, W, C):
    rng = np.random.default_rng(W)
    n = 4
    R = Ring(n, W, C, kv, d, layers=2, layer=1)
    for lengths in ([0, 1, 64, 63], [0, 60, 65, 1]):
        for r, m in enumerate(lengths):
            while m > 0:
                step = min(m, C - 63)
                x = values(rng, (1, step, kv, d), 0.5)
                R.write([r], x, -x)
                R.advance([r], step)
                m -= step
        reqs = [3, 1, 0, 2]
        k = torch.full((n, W, kv, d), 7.0, dtype=TYPE[typ], device=DEV)
        v = torch.full((n, W, kv, d), 7.0, dtype=TYPE[typ], device=DEV)
        vis, status = i32([9] * n), i32([9] * n)
        R.ring.read_kv(1, n, i32(reqs), k, v, vis, status)
        torch.cuda.synchronize()
        assert (status == 0).all()
        for i, r in enumerate(reqs):
            m = min(W, int(R.ref.length[r]))
            assert vis[i] == m
            for got, want in zip((k, v), R.ref.rows(r, int(R.ref.length[r]) - m,
                                                    int(R.ref.length[r]))):
                want = torch.from_numpy(want).float().to(TYPE[typ]).transpose(0, 1)
                assert torch.equal(got[i, :m].cpu(), want)
                assert (got[i, m:] == 7).all()


def attend(R, reqs, q, mask, count=None, scale=None, workspace=True, out=None, lse=None):
    n, nq, heads, d = q.shape
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    lse = torch.full(q.shape[:3], 7.0, device=DEV) if lse is None else lse
    status = torch.full((n,), 9, dtype=torch.int32, device=DEV)
    need = R.ring.attend_workspace(n, nq, heads)
    ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device=DEV) if workspace else None
    R.ring.attend(R.layer, n, i32(reqs), q, out, scale=scale or d ** -0.5, mask=mask,
                  count=None if count is None else i32(count), lse=lse, status=status,
                  workspace=ws[:need] if workspace else None)
    torch.cuda.synchronize()
    if workspace:
        assert (ws[need:] == 0x7F).all(), "the workspace was overrun"
    assert (status == 0).all()
    return out, lse


def check_attend(R, reqs, q, mask, out, lse, count=None, scale=None):
    n, nq, heads, d = q.shape
    kv, W = R.ref.kv, R.ref.W
    group = heads // kv
    scale = scale or d ** -0.5
    q64, out, lse = q.cpu().double().numpy(), out.cpu().double().numpy(), lse.cpu().double().numpy()
    for i, r in enumerate(reqs):
        m = nq if count is None else count[i]
        assert (out[i, m:] == 7).all() and (lse[i, m:] == 7).all(), "a padded query was written"
        for j in range(m):
            lo, hi = ref.span(mask, int(R.ref.length[r]), m, j, W)
            keys, vals = R.ref.rows(r, lo, hi)
            for h in range(kv):
                at = (i, j, slice(h * group, (h + 1) * group))
                o, s, spread, size = ref.attend(q64[at], keys[h], vals[h], scale)
                if hi == lo:
                    assert (out[at] == 0).all() and (lse[at] == -np.inf).all()
                    continue
                rows, c = hi - lo, 264
                tol = c * EPS32 * size + (rows + 16) * EPS32 + 16 * EPS32 * (1 + np.abs(s))
                err = np.abs(lse[at] - s)
                assert (err <= tol).all(), (i, j, h, (err / tol).max())
                d_p = 2 * c * EPS32 * size + 32 * EPS32
                tol = (H + d_p + 2 * rows * EPS32)[:, None] * spread + H * np.abs(o)
                err = np.abs(out[at] - o)
                assert (err <= tol).all(), (i, j, h, (err / tol).max())


def filled(seed, n, W, C, kv, d, lengths, new, layers=1, layer=0):
    """A ring with `lengths` rows kept and `new` more written."""
    rng = np.random.default_rng(seed)
    R = Ring(n, W, C, kv, d, layers, layer)
    for r, m in enumerate(lengths):
        while int(R.ref.length[r]) < m:
            step = min(C - 63, m - int(R.ref.length[r]))
            R.write([r], values(rng, (1, step, kv, d), 0.3), values(rng, (1, step, kv, d), 0.3))
            R.advance([r], step)
    if new:
        R.write(list(range(n)), values(rng, (n, new, kv, d), 0.3), values(rng, (n, new, kv, d), 0.3))
    return R


@pytest.mark.parametrize("mask", ["causal", "block", "kept"])
@pytest.mark.parametrize("d,kv,group", [(64, 1, 1), (128, 2, 4), (256, 1, 16), (64, 3, 5),
                                        (128, 1, 17)])
def test_attend_few_queries(mask, d, kv, group):
    """Requests without rows, with one, around a block, full and wrapped; one to
    five queries, and entries with fewer."""
    lengths = [0, 1, 63, 64, 65, 130, 200, 777]
    n, W, C = len(lengths), 150, 256
    for nq in (1, 2, 5):
        R = filled(nq, n, W, C, kv, d, lengths, nq)
        q = torch.randn(n, nq, kv * group, d, device=DEV).bfloat16()
        count = None if nq < 5 else [5, 0, 1, 2, 3, 4, 5, 0]
        reqs = list(range(n))
        out, lse = attend(R, reqs, q, mask, count)
        check_attend(R, reqs, q, mask, out, lse, count)


@pytest.mark.parametrize("mask", ["causal", "block"])
@pytest.mark.parametrize("d,kv,group,nq", [(64, 2, 4, 40), (128, 1, 8, 33), (256, 1, 2, 70),
                                           (128, 1, 1, 140), (64, 1, 3, 257)])
def test_attend_prompts(mask, d, kv, group, nq):
    """Chunks of a prompt: first ones (no rows kept), later ones, padded ones."""
    lengths, count = [0, 100, 1000], [nq, nq // 2, nq - 1]
    W = 200
    C = (W + nq + 63) // 64 * 64 + 64
    R = filled(nq, 3, W, C, kv, d, lengths, nq)
    q = torch.randn(3, nq, kv * group, d, device=DEV).bfloat16()
    for c in (None, count):
        out, lse = attend(R, [0, 1, 2], q, mask, c)
        check_attend(R, [0, 1, 2], q, mask, out, lse, c)


@pytest.mark.parametrize("d,n,kv,group,nq,W", [(128, 45, 4, 4, 64, 100), (128, 23, 8, 1, 256, 70),
                                               (256, 1, 1, 1, 140, 2500), (256, 3, 2, 3, 60, 130),
                                               (128, 49, 4, 4, 64, 100), (128, 25, 8, 1, 256, 70),
                                               (256, 44, 3, 3, 43, 130), (256, 1, 4, 16, 250, 2000),
                                               (256, 1, 4, 4, 320, 900)])
@pytest.mark.parametrize("mask", ["causal", "block"])
def test_attend_rows_that_share_blocks(d, n, kv, group, nq, W, mask):
    """Enough query rows for the waves of a workgroup to share each block: full ones, and
    entries with fewer rows than a workgroup, a wave or anything."""
    C = (W + nq + 63) // 64 * 64 + 64
    lengths = [(0, W // 2, W + 64 * r, 3 * W + r)[r % 4] for r in range(n)]
    count = None
    if n > 1:
        count = [(nq, 0, 1, nq // 2 + 1, nq - 1)[r % 5] for r in range(n)]
    R = filled(d + W, n, W, C, kv, d, lengths, nq)
    q = torch.randn(n, nq, kv * group, d, device=DEV).bfloat16()
    out, lse = attend(R, list(range(n)), q, mask, count)
    check_attend(R, list(range(n)), q, mask, out, lse, count)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_workspace_covers_smaller_calls(d):
    kv, W = 2, 3000
    ring = filled(d, 6, W, 3456, kv, d, [W] * 6, 1).ring
    big = (6, 300, 16)
    ws = torch.empty(ring.attend_workspace(*big), dtype=torch.uint8, device=DEV)
    for n in (1, 2, 3, 5, 6):
        for nq in (1, 2, 5, 16, 60, 150, 250, 300):
            for heads in (2, 4, 10, 16):
                q = torch.zeros(n, nq, heads, d, dtype=torch.bfloat16, device=DEV)
                for mask in ("causal", "block", "kept"):
                    ring.attend(0, n, None, q, torch.empty_like(q), scale=1.0, mask=mask,
                                workspace=ws)
                assert ring.attend_workspace(n, nq, heads) <= ws.numel()


@pytest.mark.parametrize("W,nq,n", [(1, 1, 2), (1, 5, 1), (64, 1, 1), (5000, 1, 1), (3500, 3, 3),
                                    (700, 1, 40)])
def test_attend_window_sizes(W, nq, n):
    """From a window of one token to long ones, cut into shares or not."""
    C = (W + nq + 63) // 64 * 64 + 64
    R = filled(W, n, W, C, 2, 128, [W + 11 * r for r in range(n)], nq)
    q = torch.randn(n, nq, 8, 128, device=DEV).bfloat16()
    out, lse = attend(R, list(range(n)), q, "causal")
    check_attend(R, list(range(n)), q, "causal", out, lse)


def test_attend_requests_layers_and_strides():
    """A subset of the requests in another order (one of them twice), the second of
    three layers, queries as slices of one projection, a negative scale."""
    R = filled(3, 5, 90, 192, 2, 64, [10, 300, 64, 128, 77], 2, layers=3, layer=1)
    reqs = [4, 1, 1, 0]
    wide = torch.randn(4, 2, 4, 3 * 64 + 5, device=DEV).bfloat16()
    for at in (0, 64, 3):
        q = wide[..., at:at + 64]
        for scale in (0.125, -0.3):
            out, lse = attend(R, reqs, q, "causal", scale=scale)
            check_attend(R, reqs, q, "causal", out, lse, scale=scale)
    # one query row for all
    q = wide[:1, :1, :1, :64].expand(4, 2, 4, 64)
    out, lse = attend(R, reqs, q, "causal")
    check_attend(R, reqs, q, "causal", out, lse)


def test_large_scores():
    """Scores that rise by far more than the exponent's range from block to block,
    and rows that weigh nothing."""
    rng = np.random.default_rng(11)
    R = Ring(1, 256, 384, 1, 64)
    k, v = values(rng, (1, 256, 1, 64), 0.0), values(rng, (1, 256, 1, 64), 0.0)
    k *= 2.0 ** (np.arange(256) // 40)[None, :, None, None]
    R.write([0], k, v)
    R.advance([0], 256)
    q = (8 * torch.randn(1, 3, 4, 64, device=DEV)).bfloat16()
    out, lse = attend(R, [0], q, "kept")
    check_attend(R, [0], q, "kept", out, lse)


def test_a_scale_of_zero():
    """Every row seen weighs the same; rows left out still weigh nothing."""
    R = filled(12, 3, 100, 192, 1, 64, [0, 30, 150], 2)
    q = torch.randn(3, 2, 2, 64, device=DEV).bfloat16()
    out = torch.zeros_like(q)
    lse = torch.zeros(3, 2, 2, device=DEV)
    ws = torch.zeros(R.ring.attend_workspace(3, 2, 2), dtype=torch.uint8, device=DEV)
    R.ring.attend(0, 3, None, q, out, scale=0.0, lse=lse, workspace=ws)
    for r, m in enumerate([0, 30, 150]):
        for j in range(2):
            lo, hi = ref.span("causal", m, 2, j, 100)
            v = R.ref.rows(r, lo, hi)[1][0]
            got = out[r, j].double().cpu().numpy()
            # weights of 1, exact in bf16; sums of 100 values and the output's rounding
            assert (np.abs(got - v.mean(0)) <= H * np.abs(v.mean(0)) + 128 * EPS32 *
                    np.abs(v).mean(0)).all()
            assert (lse[r, j].cpu() - np.log(hi - lo)).abs().max() <= 16 * EPS32 * (1 + np.log(100))


def test_rows_overwritten_after_a_rollback():
    """A query that would see a row that a dropped one has overwritten: the entry is
    refused, the others are not."""
    W, C = 100, 128
    R = filled(4, 2, W, C, 1, 64, [300, 300], 25)
    R.advance([0, 1], 25)
    R.rollback([0], [301])  # high 325, its rows from 201 on lie in slots still theirs
    rng = np.random.default_rng(4)
    R.write([0, 1], values(rng, (2, 2, 1, 64)), values(rng, (2, 2, 1, 64)))
    q = torch.randn(2, 2, 2, 64, device=DEV).bfloat16()
    out, lse = attend(R, [0, 1], q, "causal")
    check_attend(R, [0, 1], q, "causal", out, lse)
    # kept length forced below the limit of a rollback
    R.length[0] = R.ref.length[0] = 290
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    status = i32([9, 9])
    ws = torch.zeros(R.ring.attend_workspace(2, 2, 2), dtype=torch.uint8, device=DEV)
    R.ring.attend(0, 2, None, q, out, scale=0.125, lse=lse, status=status, workspace=ws)
    torch.cuda.synchronize()
    assert status.tolist() == [-2, 0]
    assert (out[0] == 7).all() and (lse[0] == 7).all()
    check_attend(R, [1], q[1:], "causal", out[1:], lse[1:])


def test_status_of_bad_entries():
    """Requests and counts out of range, lengths that are no lengths: such entries
    write nothing, the others go on."""
    from hierarchical_sparse_kv_resolve_amd import kvr
    R = filled(5, 6, 64, 192, 1, 64, [70] * 6, 0)
    reqs = i32([-1, 6, 2, 3, 4, 5])
    count = i32([1, 1, 3, -1, 1, 1])
    R.length[4] = -3
    R.high[5] = 60
    before = [x.clone() for x in (R.codes, R.scales, R.length, R.high)]
    k = torch.ones(6, 2, 1, 64, device=DEV)
    want = [kvr.E_ARG] * 4 + [kvr.E_STATE] * 2
    status = i32([9] * 6)
    R.ring.write_kv(0, 6, reqs, k, k, count, status)
    assert status.tolist() == want
    R.ring.advance(6, reqs, 2, count, status.fill_(9))
    assert status.tolist() == want
    q = torch.zeros(6, 2, 1, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 7.0)
    ws = torch.zeros(R.ring.attend_workspace(6, 2, 1), dtype=torch.uint8, device=DEV)
    R.ring.attend(0, 6, reqs, q, out, scale=0.1, count=count, status=status.fill_(9), workspace=ws)
    assert status.tolist() == want
    rows = torch.full((6, 64, 1, 64), 7.0, device=DEV)
    R.ring.read_kv(0, 6, reqs, rows, rows.clone(), status=status.fill_(9))
    assert status.tolist() == [kvr.E_ARG] * 2 + [0] * 2 + [kvr.E_STATE] * 2
    assert (rows[[0, 1, 4, 5]] == 7).all() and (out == 7).all()
    for x, y in zip((R.codes, R.scales, R.length, R.high), before):
        assert torch.equal(x, y)
    # positions at the end of the range
    R.length[2] = R.high[2] = 2 ** 31 - 66
    R.ring.advance(1, i32([2]), 2, None, status.fill_(9))
    assert status[0] == kvr.E_CAPACITY and R.length[2] == 2 ** 31 - 66
    R.ring.advance(1, i32([2]), 1, None, status.fill_(9))
    assert status[0] == 0 and R.length[2] == 2 ** 31 - 65


def test_far_positions():
    """Lengths near the end of the range: slots, masks and block ends hold."""
    R = Ring(1, 100, 192, 1, 64)
    start = (2 ** 31 - 65 - 300) // 64 * 64
    R.codes.zero_()
    R.scales.fill_(27)
    for x in (R.length, R.high):
        x.fill_(start)
    R.ref.length[0] = R.ref.high[0] = start
    rng = np.random.default_rng(2)
    for rows in (120, 100, 60):
        k = values(rng, (1, rows, 1, 64))
        R.write([0], k, -k)
        R.advance([0], rows)
    R.write([0], k[:, :4], k[:, :4])
    q = torch.randn(1, 4, 3, 64, device=DEV).bfloat16()
    out, lse = attend(R, [0], q, "causal")
    check_attend(R, [0], q, "causal", out, lse)


def test_layers_past_32_bits():
    """The last of layers that hold more than 4 GiB of codes together."""
    n, C, kv, d = 4, 8192, 8, 256
    layers = 41
    codes = torch.zeros(layers, n, C // 64, kv, 2, 64 * d, dtype=torch.uint8, device=DEV)
    assert codes.numel() > 5 << 30
    scales = torch.full((layers, n, C // 64, kv, 2), 127, dtype=torch.uint8, device=DEV)
    from hierarchical_sparse_kv_resolve_amd import DraftRing
    length, high = i32([8000] * n), i32([8000] * n)
    ring = DraftRing(n, 64, C, 0, None, length, high)
    ring.bind_kv(layers, kv, d, codes, scales)
    k = torch.randn(n, 3, kv, d, device=DEV).bfloat16()
    ring.write_kv(layers - 1, n, None, k, k)
    ring.advance(n, None, 3)
    out_k = torch.zeros(n, 64, kv, d, device=DEV)
    out_v = torch.zeros_like(out_k)
    ring.read_kv(layers - 1, n, None, out_k, out_v)
    assert torch.equal(out_k, out_v) and (out_k[:, :61] == 0).all()
    # a code is off by at most half a step: 2^-4, or 2^-10 of its scale (at most 2^-6 here)
    err = (out_k[:, 61:] - k.float()).abs()
    assert (err <= (k.float().abs() * 2.0 ** -4).clamp(min=2.0 ** -16)).all()
    assert (codes[:-1].view(torch.int64) == 0).all()
    ring.write_kv(layers - 1, n, None, k, k)
    q = torch.randn(n, 1, kv, d, device=DEV).bfloat16()
    out = torch.zeros_like(q)
    ws = torch.zeros(ring.attend_workspace(n, 1, kv), dtype=torch.uint8, device=DEV)
    ring.attend(layers - 1, n, None, q, out, scale=1 / 16, workspace=ws)
    rows = torch.cat([out_k[:, 1:], out_k[:, 61:62]], 1).transpose(1, 2).double()  # [n, kv, 64, d]
    s = (q.double()[:, 0, :, None] * rows).sum(-1) / 16
    want = (torch.softmax(s, -1)[..., None] * rows).sum(2)
    spread = (torch.softmax(s, -1)[..., None] * rows.abs()).sum(2)
    # as above, with d_p of scores below 64 in size
    assert ((out[:, 0].double() - want).abs() <= (H + 2e-3) * spread + H * want.abs()).all()


def test_two_calls_at_once():
    """Two layers on two streams, each with its own workspace."""
    R = filled(6, 4, 3500, 3648, 2, 128, [3600] * 4, 1, layers=2, layer=0)
    R.codes[1], R.scales[1] = R.codes[0], R.scales[0]
    q = torch.randn(4, 1, 16, 128, device=DEV).bfloat16()
    want, want_lse = attend(R, [0, 1, 2, 3], q, "causal")
    need = R.ring.attend_workspace(4, 1, 16)
    assert need > 0
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(q) for _ in range(2)]
    ws = [torch.zeros(need, dtype=torch.uint8, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for l in range(2):
            R.ring.attend(l, 4, None, q, outs[l], scale=128 ** -0.5, workspace=ws[l],
                          stream=streams[l])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_captured_and_replayed():
    """A step's write, attention and advance in one graph, replayed with new
    contents beside an eager ring."""
    n, kv, d, W, C = 3, 2, 64, 700, 832
    A, B = (filled(7, n, W, C, kv, d, [650, 3, 64], 0) for _ in range(2))
    k = torch.randn(n, 2, kv, d, device=DEV).bfloat16()
    q = torch.randn(n, 2, 8, d, device=DEV).bfloat16()
    count = i32([2, 1, 0])
    need = A.ring.attend_workspace(n, 2, 8)

    def step(R, out, lse, ws):
        R.ring.write_kv(0, n, None, k, k, count)
        R.ring.attend(0, n, None, q, out, scale=0.2, count=count, lse=lse, workspace=ws)
        R.ring.advance(n, None, 2, count)

    bufs = [(torch.zeros_like(q), torch.zeros(n, 2, 8, device=DEV),
             torch.zeros(need, dtype=torch.uint8, device=DEV)) for _ in range(2)]
    step(A, *bufs[0])
    step(B, *bufs[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(A, *bufs[0])
    for _ in range(70):
        k.copy_(torch.randn_like(k, dtype=torch.float32))
        q.copy_(torch.randn_like(q, dtype=torch.float32))
        count.copy_(torch.randint(0, 3, (n,), device=DEV))
        g.replay()
        step(B, *bufs[1])
        torch.cuda.synchronize()
        for a, b in zip(bufs[0][:2], bufs[1][:2]):
            assert torch.equal(a, b)
        for a, b in ((A.codes, B.codes), (A.scales, B.scales), (A.length, B.length),
                     (A.high, B.high)):
            assert torch.equal(a, b)


def test_same_results_every_time():
    for W, nq in ((1000, 1), (3000, 1), (300, 40)):
        R = filled(9, 2, W, (W + 191) // 64 * 64, 1, 128, [2 * W, W - 100], nq)
        q = torch.randn(2, nq, 16, 128, device=DEV).bfloat16()
        first = attend(R, [0, 1], q, "causal")
        for _ in range(5):
            again = attend(R, [0, 1], q, "causal")
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_refusals():
    from hierarchical_sparse_kv_resolve_amd import DraftRing, KvrError
    R = filled(10, 2, 64, 192, 2, 64, [70, 70], 0)
    k = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16, device=DEV)

    def refused(call, error, match, good, **kw):
        with pytest.raises(error, match=match):
            call(**{**good, **kw})

    good = dict(layer=0, n=2, req_ids=None, k=k, v=k)
    R.ring.write_kv(**good)
    w = R.ring.write_kv
    refused(w, KvrError, r"layer 1 outside", good, layer=1)
    refused(w, KvrError, "request count 3", good, n=3, k=torch.cat([k, k[:1]]),
            v=torch.cat([k, k[:1]]))
    refused(w, ValueError, "k: shape", good, k=k[..., :32])
    refused(w, ValueError, "v: shape", good, v=k[:, :, :1])
    refused(w, TypeError, "v: expected bfloat16", good, v=k.float())
    refused(w, TypeError, "k: expected bfloat16 or", good, k=k.double())
    refused(w, TypeError, "GPU tensor", good, k=k.cpu())
    refused(w, ValueError, "dimensions", good, k=k[0])
    refused(w, ValueError, "last dimension", good,
            k=torch.zeros(2, 1, 64, 2, dtype=torch.bfloat16, device=DEV).transpose(2, 3))
    refused(w, TypeError, "count: expected int32", good, count=torch.zeros(2, device=DEV))
    big = torch.zeros(2, 130, 2, 64, dtype=torch.bfloat16, device=DEV)
    refused(w, KvrError, r"rows must be in \[0, capacity - 63\]", good, k=big, v=big)

    rows = torch.zeros(2, 64, 2, 64, device=DEV)
    good = dict(layer=0, n=2, req_ids=None, k=rows, v=rows.clone())
    R.ring.read_kv(**good)
    refused(R.ring.read_kv, ValueError, "k: shape", good, k=rows[:, :63])
    refused(R.ring.read_kv, ValueError, "not contiguous", good,
            v=torch.zeros(2, 64, 2, 65, device=DEV)[..., :64])

    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(R.ring.attend_workspace(2, 3, 4) + 16, dtype=torch.uint8, device=DEV)
    good = dict(layer=0, n=2, req_ids=None, q=q, out=torch.zeros_like(q), scale=0.1, workspace=ws)
    a = R.ring.attend
    a(**good)
    refused(a, ValueError, "unknown mask", good, mask="full")
    refused(a, TypeError, "q: expected bfloat16", good, q=q.half())
    refused(a, ValueError, "out: shape", good, out=q[:, :2])
    refused(a, ValueError, "lse: shape", good, lse=torch.zeros(2, 4, device=DEV))
    odd = torch.zeros(2, 3, 5, 64, dtype=torch.bfloat16, device=DEV)
    refused(a, KvrError, "multiple of the K/V heads", good, q=odd, out=odd.clone())
    many = torch.zeros(2, 130, 4, 64, dtype=torch.bfloat16, device=DEV)
    refused(a, KvrError, "130 causal queries: the ring keeps the rows of 129", good, q=many,
            out=many.clone())
    wide = torch.zeros(2, 193, 4, 64, dtype=torch.bfloat16, device=DEV)
    refused(a, KvrError, "193 new tokens", good, q=wide, out=wide.clone(), mask="block")
    flat = torch.zeros(q.numel() + 8, dtype=torch.bfloat16, device=DEV)
    refused(a, KvrError, "not aligned", good, out=flat[4:-4].view(q.shape))
    for scale in (float("nan"), float("inf"), -float("inf"), 2.0 ** 127):
        refused(a, KvrError, "scale must be finite", good, scale=scale)
    R2 = filled(10, 1, 8000, 8128, 1, 64, [8000], 1)
    q1 = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    refused(R2.ring.attend, KvrError, "the workspace has 0 bytes", dict(
        layer=0, n=1, req_ids=None, q=q1, out=torch.zeros_like(q1), scale=0.1))

    # rings without one or the other part
    rows = torch.zeros(2, 64, dtype=torch.uint8, device=DEV)
    with pytest.raises(KvrError, match="holds no rows"):
        R.ring.append(2, None, 1, rows)
    with pytest.raises(KvrError, match="holds no rows"):
        R.ring.window(2, None, rows)
    ring = torch.zeros(2, 100, 16, dtype=torch.uint8, device=DEV)
    plain = DraftRing(2, 64, 100, 16, ring, R.length, R.high)
    with pytest.raises(KvrError, match="not a multiple of 64"):
        plain.bind_kv(1, 1, 64, R.codes, R.scales)
    with pytest.raises(KvrError, match="no K/V layers"):
        plain.attend_workspace(1, 1, 1)
    with pytest.raises(KvrError, match="no K/V layers"):
        plain.d_head, plain.kv_heads = 64, 2
        plain.write_kv(0, 2, None, k, k)
    fresh = DraftRing(2, 64, 192, 0, None, R.length, R.high)
    for args in ((0, 1, 64), (1, 0, 64), (1, 257, 64), (1, 1, 96)):
        with pytest.raises(KvrError, match="d_head 64"):
            fresh.bind_kv(*args, torch.zeros(1 << 24, dtype=torch.uint8, device=DEV),
                          torch.zeros(1 << 16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="codes: "):
        fresh.bind_kv(2, 2, 64, R.codes, R.scales)
