"""Two calls at once, each on its own stream with its own inputs, outputs and
workspace, all of them enqueued before the one wait: what a call gives alone, which
is compared with the 64-bit forms, it gives beside the other."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import test_gpu_logprob as lp
from tests.test_gpu_draft_kv import DEV, Ring, attend, check_attend, values

pytestmark = pytest.mark.gpu
ROUNDS = 25


def both(calls):
    """calls[i](stream, round), alternating."""
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for r in range(ROUNDS):
        for call, s in zip(calls, streams):
            call(s, r)
    torch.cuda.synchronize()


@pytest.mark.parametrize("d,n,nq,W,sizes", [(128, 4, 1, 3500, True), (64, 2, 3, 6000, True),
                                            (256, 1, 250, 1000, True), (128, 8, 130, 300, False)])
def test_attention_of_two_layers(d, n, nq, W, sizes):
    """Shares in workspaces or none, rows of few queries and of many."""
    kv, heads, C = 2, 16, (W + nq + 127) // 64 * 64 + 64
    rings, rng = [], np.random.default_rng(d)
    lengths = [W + 61 * r for r in range(n)]
    for layer in range(2):  # other keys and values in each layer of one ring
        R = Ring(n, W, C, kv, d, 2, layer)
        if layer:
            R.ring, R.codes, R.scales = rings[0].ring, rings[0].codes, rings[0].scales
            R.length, R.high = rings[0].length, rings[0].high
        rings.append(R)
    for r, m in enumerate(lengths):
        while int(rings[0].ref.length[r]) < m:
            step = min(C - 63, m - int(rings[0].ref.length[r]))
            for R in rings:
                R.write([r], values(rng, (1, step, kv, d), 0.3), values(rng, (1, step, kv, d), 0.3))
            rings[0].advance([r], step)
            rings[1].ref.advance(r, step)
    for R in rings:
        R.write(list(range(n)), values(rng, (n, nq, kv, d), 0.3), values(rng, (n, nq, kv, d), 0.3))
    q = [torch.randn(n, nq, heads, d, device=DEV).bfloat16() for _ in rings]
    want = [attend(R, list(range(n)), x, "causal") for R, x in zip(rings, q)]
    for R, x, w in zip(rings, q, want):
        few = slice(0, 4)  # (all queries of the others are compared bit for bit)
        check_attend(R, list(range(n))[few], x[few], "causal", w[0][few], w[1][few])
    assert not torch.equal(want[0][0], want[1][0])
    need = rings[0].ring.attend_workspace(n, nq, heads)
    assert (need > 0) or not sizes
    outs = [[(torch.zeros_like(x), torch.zeros(x.shape[:3], device=DEV)) for _ in range(ROUNDS)]
            for x in q]
    ws = [torch.full((need,), 0x7F, dtype=torch.uint8, device=DEV) for _ in q]

    def one(layer):
        return lambda s, r: rings[0].ring.attend(layer, n, None, q[layer], outs[layer][r][0],
                                                 scale=d ** -0.5, lse=outs[layer][r][1],
                                                 workspace=ws[layer], stream=s)

    both([one(0), one(1)])
    for layer in range(2):
        for out, lse in outs[layer]:
            assert torch.equal(out, want[layer][0]) and torch.equal(lse, want[layer][1])


@pytest.mark.parametrize("n,vocab,top", [(9, 50000, 20), (64, 131072, 64), (1, 131072, 5)])
def test_log_probabilities_of_two_batches(n, vocab, top):
    rng = np.random.default_rng(vocab + top)
    ctx = lp.context()
    x = [lp.rows(rng, n, vocab, "bf16") for _ in range(2)]
    tokens = [torch.from_numpy(rng.integers(0, vocab, (n, 3)).astype(np.int32)).to(DEV)
              for _ in range(2)]
    want = [lp.call(a, b, top, 1.25, ctx) for a, b in zip(x, tokens)]
    for a, b, w in zip(x, tokens, want):
        few = slice(0, 3)
        lp.check(a[few], b[few], top, 1.25, {k: v[few] for k, v in w.items()})
    outs = [[{k: torch.full_like(v, 7) for k, v in w.items()} for _ in range(ROUNDS)] for w in want]
    ws = [torch.full((ctx.logprob_workspace(n, vocab),), 0x7F, dtype=torch.uint8, device=DEV)
          for _ in range(2)]

    def one(i):
        def call(s, r):
            o = outs[i][r]
            ctx.token_logprobs(n, x[i], tokens[i], o["logprob"], lse=o["lse"], entropy=o["entropy"],
                               top_ids=o["top_ids"], top_logprob=o["top_logprob"], scale=1.25,
                               workspace=ws[i], stream=s)
        return call

    both([one(0), one(1)])
    for i in range(2):
        assert not torch.equal(want[i]["lse"], want[1 - i]["lse"])
        for o in outs[i]:
            assert all(torch.equal(o[k], want[i][k]) for k in o)
