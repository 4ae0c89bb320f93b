"""The drafter's window in 8 bits at its edges: windows shorter than a block after
rollbacks that dropped tokens have wrapped past, values at the top of the types'
range, windows whose rows are gone.  Codes and scales bit for bit, as
in test_gpu_draft_kv.py (no tolerance); attention by that file's bounds."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_draft_kv import DEV, TYPE, Ring, attend, check_attend, filled, i32, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("typ", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("W,C,d", [(16, 64, 64), (1, 128, 64), (17, 128, 128), (62, 128, 64),
                                   (63, 128, 64), (30, 192, 256)])
def test_dropped_rows_that_wrapped_into_the_block(W, C, d, typ):
    """Dropped tokens far larger than the kept ones lie in slots of the block that is
    written next, up to the rollback's limit: those slots become 0, and the scale
    follows the rows kept and the new ones alone."""
    rng = np.random.default_rng(W * d)
    kv, big = 2, 2.0 ** 8
    R = Ring(2, W, C, kv, d)

    def put(reqs, rows, size):
        while rows > 0:
            step = min(rows, C - 63)
            x = np.clip(values(rng, (len(reqs), step, kv, d), 0.3), -50, 50)
            R.write(reqs, x * size, -x[..., ::-1].copy() * size, typ=typ)
            R.advance(reqs, step)
            rows -= step

    for r, kept in enumerate((C + 36, 2 * C + 63)):
        put([r], kept, 1 / big)
        put([r], C - W, big)  # drafted and rejected
        R.rollback([r], [kept])
    for rows in (1, 1, min(5, C - 63), 1):
        x = values(rng, (2, rows, kv, d), 0.3) / big
        R.write([0, 1], x, -x, typ=typ)
        R.check()
        assert (R.ref.exp[:, :, :, :].min((1, 2, 3)) < -5).all()
        nq = min(rows, C - W + 1)
        q = torch.randn(2, nq, 3 * kv, d, device=DEV).bfloat16()
        out, lse = attend(R, [0, 1], q, "causal")
        check_attend(R, [0, 1], q, "causal", out, lse)
        R.advance([0, 1], rows)


@pytest.mark.parametrize("typ", ["bf16", "f32"])
def test_values_at_the_top_of_the_range(typ):
    """Magnitudes whose nearest code would stand for 2^128 take the one below it, 240 *
    2^120: rows read back are finite, and so are queries that do not see them."""
    rng = np.random.default_rng(9)
    kv, d, W, C = 2, 64, 64, 192
    R = Ring(1, W, C, kv, d)
    most, tie = torch.finfo(TYPE[typ]).max, 248 * 2.0 ** 120
    hold = lambda x: np.where(np.isfinite(x) & (np.abs(x) >= tie),  # noqa: E731
                              np.sign(x) * 240 * 2.0 ** 120, x)
    write = R.ref.write
    R.ref.write = lambda r, k, v: write(r, hold(k), hold(v))
    k, v = values(rng, (1, 100, kv, d), 0.3), values(rng, (1, 100, kv, d), 0.3)
    v[0, 70, 1, :6] = most, -most, tie, 247 * 2.0 ** 120, -2.0 ** 127, 1.0
    v[0, 71, 0, 5] = np.inf  # (its neighbours of that token stay values)
    v[0, 71, 0, 6] = -most
    k[0, 99, 0, :2] = -most, 232 * 2.0 ** 120
    R.write([0], k, v, typ=typ)
    R.check()
    q = torch.randn(1, 70, 4 * kv, d, device=DEV).bfloat16()
    out, lse = attend(R, [0], q, "causal")  # positions 0 to 69, in the block of the 70th
    check_attend(R, [0], q, "causal", out, lse)
    R.advance([0], 100)
    x = values(rng, (1, 1, kv, d))
    R.write([0], x, x, typ=typ)  # as rows kept
    R.check()
    R.advance([0], 1)
    got = torch.zeros(1, W, kv, d, device=DEV), torch.zeros(1, W, kv, d, device=DEV)
    R.ring.read_kv(0, 1, None, *got)
    for a, b in zip(got, R.ref.rows(0, 101 - W, 101)):
        b = torch.from_numpy(b).float().transpose(0, 1)
        nan = a[0].cpu().isnan()
        assert torch.equal(nan, b.isnan()) and torch.equal(a[0].cpu()[~nan], b[~nan])
        assert (a[0][~a[0].isnan()].abs() <= 240 * 2.0 ** 120).all()


def test_read_back_of_overwritten_rows():
    """A window that reaches below the oldest position the ring still holds is refused;
    one that ends there is not, and neither are the other entries."""
    from hierarchical_sparse_kv_resolve_amd import kvr
    W, C = 100, 192
    R = filled(3, 3, W, C, 1, 64, [300, 300, 300], 0)
    for length, want in ((300, 0), (208, 0), (207, kvr.E_RANGE), (120, kvr.E_RANGE)):
        R.length[1] = length  # below a rollback's limit, 208, from 207 on
        k, v = (torch.full((3, W, 1, 64), 7.0, device=DEV) for _ in range(2))
        vis, status = i32([9] * 3), i32([9] * 3)
        R.ring.read_kv(0, 3, None, k, v, vis, status)
        torch.cuda.synchronize()
        assert status.tolist() == [0, want, 0]
        assert vis.tolist() == [W, 9 if want else W, W]
        for r in range(3):
            end = length if r == 1 else 300
            if r == 1 and want:
                assert (k[r] == 7).all() and (v[r] == 7).all()
                continue
            for got, x in zip((k, v), R.ref.rows(r, end - W, end)):
                assert torch.equal(got[r].cpu(), torch.from_numpy(x).float().transpose(0, 1))
