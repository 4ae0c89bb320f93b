"""The drafter's window in 8 bits at its edges: windows shorter than a block after
rollbacks that dropped tokens have wrapped past.  Codes and scales bit for bit, as
in test_gpu_draft_kv.py (no tolerance); attention by that file's bounds."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_draft_kv import DEV, Ring, attend, check_attend, values

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
