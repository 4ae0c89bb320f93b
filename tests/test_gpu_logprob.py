"""Log probabilities of tokens, entropy and alternatives against a plain 64-bit form.

Tolerances.  eps = 2^-24.  A probability's exponent d = f (x - m) is off by 3 eps
|d| (difference, f, product), hardware exp2 by a few eps; terms with |d| > 40
weigh below e^-40.  So each term is off by (3 * 40 + 8) eps relative, sums of
vocab terms (at most 64 a thread in turn, then trees) by 96 eps more, the
logarithm's result by that and 8 eps of itself: ln l is off by
  L = 256 eps (1 + ln l).
lse = scale m + ln l and logprob = scale (x - m) - ln l add 2 roundings each:
|.| errors at most L + 3 eps (|value| + |scale m|).  entropy = ln l + u / l, terms
of one sign: off by 2 L + 256 eps entropy + 128 eps (1 + entropy) <= 4 L + 512 eps
(1 + entropy).  Tokens are exact: compared as they are."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
TYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"


def context():
    from hierarchical_sparse_kv_resolve_amd import Context
    return Context(n_req=1, n_layers=1, history_rows=0, max_new_rows=1, page_rows=1, tail_rows=0,
                   hot_slots=1, row_bytes=16, sel_cap=1, pool_pages=0)


def call(logits, tokens=None, top=0, scale=1.0, ctx=None, stream=None, ws=None):
    n, vocab = logits.shape
    ctx = ctx or context()
    f = lambda *s: torch.full(s, 7.0, device=DEV)  # noqa: E731
    m = 0 if tokens is None else tokens.shape[1]
    out = dict(logprob=f(n, m) if tokens is not None else None, lse=f(n), entropy=f(n),
               top_ids=torch.full((n, top), 7, dtype=torch.int32, device=DEV) if top else None,
               top_logprob=f(n, top) if top else None)
    need = ctx.logprob_workspace(n, vocab)
    buf = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device=DEV) if ws is None else ws
    if stream is not None:  # the outputs are filled on the current stream
        stream.wait_stream(torch.cuda.current_stream())
    ctx.token_logprobs(n, logits, tokens, out["logprob"], lse=out["lse"], entropy=out["entropy"],
                       top_ids=out["top_ids"], top_logprob=out["top_logprob"], scale=scale,
                       workspace=buf, stream=stream)
    torch.cuda.synchronize()
    assert ws is not None or (buf[need:] == 0x7F).all(), "the workspace was overrun"
    return out


def check(logits, tokens, top, scale, out):
    x = logits.cpu().double().numpy()
    n, vocab = x.shape
    got = {k: None if v is None else v.cpu().numpy() for k, v in out.items()}
    for i in range(n):
        row = x[i]
        # the lower token first among equals
        order = np.argsort(-row, kind="stable") if top else []
        if np.isnan(row).any() or (row == np.inf).any():
            for k in ("lse", "entropy"):
                assert np.isnan(got[k][i])
            if tokens is not None:
                assert np.isnan(got["logprob"][i]).all()
            if top:
                assert (got["top_ids"][i] == -1).all() and np.isnan(got["top_logprob"][i]).all()
            continue
        m = row.max()
        if m == -np.inf:
            assert got["lse"][i] == -np.inf and got["entropy"][i] == 0
            if tokens is not None:
                assert (got["logprob"][i] == -np.inf).all()
            if top:
                assert (got["top_ids"][i] == -1).all() and (got["top_logprob"][i] == -np.inf).all()
            continue
        t = scale * (row - m)
        e = np.exp(t)
        ln_l = np.log(e.sum())
        L = 256 * EPS * (1 + ln_l)
        lse = scale * m + ln_l
        assert abs(got["lse"][i] - lse) <= L + 3 * EPS * (abs(lse) + abs(scale * m))
        ent = ln_l - (e * np.where(e > 0, t, 0)).sum() / e.sum()
        assert abs(got["entropy"][i] - ent) <= 4 * L + 512 * EPS * (1 + ent), (i, ent)

        def close(g, ids):
            ok = (ids >= 0) & (ids < vocab)
            want = np.where(ok, t[np.where(ok, ids, 0)] - ln_l, -np.inf)
            same = g == want
            with np.errstate(invalid="ignore"):
                return (same | (np.abs(g - want) <= L + 3 * EPS * np.abs(want))).all()

        if tokens is not None:
            assert close(got["logprob"][i], tokens[i].cpu().numpy())
        if top:
            k = min(top, int((row > -np.inf).sum()))
            assert np.array_equal(got["top_ids"][i, :k], order[:k]), i
            assert (got["top_ids"][i, k:] == -1).all()
            assert (got["top_logprob"][i, k:] == -np.inf).all()
            assert close(got["top_logprob"][i, :k], order[:k])


def rows(rng, n, vocab, typ, likely=20):
    x = rng.standard_normal((n, vocab)) * 2
    at = rng.integers(0, vocab, (n, likely))
    np.put_along_axis(x, at, 6 + 4 * rng.standard_normal((n, likely)), 1)
    return torch.from_numpy(x).to(TYPE[typ]).to(DEV)


@pytest.mark.parametrize("typ", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,vocab", [(1, 1), (3, 2), (2, 7), (5, 8), (4, 63), (3, 1000), (2, 2047),
                                     (2, 2048), (1, 2049), (7, 32001), (1, 131072), (3, 100277),
                                     (1030, 300)])
def test_rows(typ, n, vocab):
    rng = np.random.default_rng(vocab + n)
    x = rows(rng, n, vocab, typ)
    tokens = torch.from_numpy(rng.integers(0, vocab, (n, 3)).astype(np.int32)).to(DEV)
    for top, scale in ((0, 1.0), (1, 0.5), (20, 1.25), (64, 3.0)):
        check(x, tokens, top, scale, call(x, tokens, top, scale))
    check(x, None, 5, 1.0, call(x, None, 5))


@pytest.mark.parametrize("typ", ["bf16", "f32"])
def test_tokens_out_of_range_and_many(typ):
    rng = np.random.default_rng(1)
    x = rows(rng, 2, 500, typ)
    for m in (64, 65, 900):
        tokens = torch.from_numpy(rng.integers(-3, 503, (2, m)).astype(np.int32)).to(DEV)
        for top in (0, 3):
            check(x, tokens, top, 1.0, call(x, tokens, top))


@pytest.mark.parametrize("typ", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lowest", [False, True])
def test_masked_logits(typ, lowest):
    """Rows with all, all but one, or most logits banned, by -infinity or the type's
    lowest value."""
    rng = np.random.default_rng(2)
    vocab = 5000
    ban = torch.finfo(TYPE[typ]).min if lowest else -np.inf
    x = rows(rng, 6, vocab, typ)
    x[0] = ban
    x[1] = ban
    x[1, 4321] = 0.5
    keep = torch.rand(vocab, device=DEV) < 0.002
    x[2, ~keep] = ban
    x[3, 100:] = ban
    x[4, :4990] = ban
    x[5, 1::2] = ban
    tokens = torch.tensor([[0, 4321, 50]] * 6, dtype=torch.int32, device=DEV)
    for scale in (1.0, 0.5):
        check(x, tokens, 20, scale, call(x, tokens, 20, scale))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_that_are_not_finite(bad):
    """They show in their own row only, wherever they stand."""
    rng = np.random.default_rng(3)
    x = rows(rng, 5, 20000, "bf16")
    for i, at in enumerate((0, 12345, 19999)):
        x[i, at] = bad
    x[1, 5:9] = -float("inf")
    x[2, :19999] = -float("inf")  # nothing but the bad one
    tokens = torch.zeros(5, 1, dtype=torch.int32, device=DEV)
    check(x, tokens, 8, 1.0, call(x, tokens, 8))


@pytest.mark.parametrize("typ", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [64, 5000, 70001])
def test_ties(typ, vocab):
    """Equal logits: all of them, many at the top, and signed zeros."""
    x = torch.zeros(5, vocab, device=DEV)
    x[1, ::3] = 2.0
    x[2, vocab // 2:] = -1.0
    x[3, 1::2] = -0.0
    x[4] = (torch.arange(vocab, device=DEV) % 7).float()
    x = x.to(TYPE[typ])
    for top in (1, 20, 64):
        check(x, None, top, 1.0, call(x, None, top))


def test_large_logits_in_one_group():
    """Many more large logits in one lane's pieces than alternatives asked for, and
    more than the list of the usual way holds."""
    rng = np.random.default_rng(4)
    vocab = 131072
    x = rows(rng, 3, vocab, "f32")
    lane = (torch.arange(vocab, device=DEV) // 8) % 64
    x[0, lane == 5] += 100.0
    x[1, (lane == 5) & (torch.arange(vocab, device=DEV) % 8 == 1)] += 100.0
    x[2] = torch.arange(vocab, device=DEV).float() / 1000
    for top in (2, 64):
        check(x, None, top, 1.0, call(x, None, top))


@pytest.mark.parametrize("typ", ["bf16", "f32"])
def test_strided_rows(typ):
    """Slices of wider rows at any offset, and one row for all."""
    rng = np.random.default_rng(5)
    wide = rows(rng, 4, 3100, typ)
    tokens = torch.zeros(4, 1, dtype=torch.int32, device=DEV)
    for at, vocab in ((0, 3100), (8, 3000), (1, 3000), (3, 2999)):
        x = wide[:, at:at + vocab]
        check(x, tokens, 5, 1.0, call(x, tokens, 5))
    x = wide[:1].expand(4, 3100)
    check(x, tokens, 5, 1.0, call(x, tokens, 5))


def test_sharp_and_flat_rows():
    """Probabilities near 1 and near 1 / vocab."""
    x = torch.zeros(3, 50000, device=DEV)
    x[0, 77] = 60.0
    x[1, 77] = 16.0
    tokens = torch.tensor([[77, 3]] * 3, dtype=torch.int32, device=DEV)
    for scale in (1.0, 5.0, 0.01):
        check(x, tokens, 2, scale, call(x, tokens, 2, scale))


def test_rows_past_32_bits():
    vocab = 131072
    n = (5 << 30) // (2 * vocab)
    x = torch.full((n, vocab), -3.0, dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(6)
    ends = torch.tensor([0, n // 2, n - 1], device=DEV)
    x[ends] = rows(rng, 3, vocab, "bf16")
    tokens = torch.zeros(n, 1, dtype=torch.int32, device=DEV)
    out = call(x, tokens, 4)
    check(x[ends], tokens[ends], 4, 1.0, {k: v[ends] for k, v in out.items()})


def test_streams_graph_and_repeats():
    """Two calls at once, a captured one replayed, the same result every time."""
    rng = np.random.default_rng(7)
    ctx = context()
    x = rows(rng, 9, 50000, "bf16")
    tokens = torch.zeros(9, 1, dtype=torch.int32, device=DEV)
    want = call(x, tokens, 20, ctx=ctx)
    need = ctx.logprob_workspace(9, 50000)
    for s in [torch.cuda.Stream() for _ in range(2)]:
        got = call(x, tokens, 20, ctx=ctx, stream=s)
        assert all(torch.equal(got[k], want[k]) for k in want)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    out = {k: torch.zeros_like(v) for k, v in want.items()}

    def one(o, w):
        ctx.token_logprobs(9, x, tokens, o["logprob"], lse=o["lse"], entropy=o["entropy"],
                           top_ids=o["top_ids"], top_logprob=o["top_logprob"], workspace=w)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one(out, ws)
    for _ in range(4):
        x.copy_(rows(rng, 9, 50000, "bf16"))
        g.replay()
        want = call(x, tokens, 20, ctx=ctx)
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want)
    ctx.timing_begin(8)
    one(out, ws)
    assert {k for k, _ in ctx.timing_end()} == {"logprob"}


def test_refusals():
    from hierarchical_sparse_kv_resolve_amd import KvrError
    c = context()
    x = torch.zeros(2, 100, device=DEV)
    tokens = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
    lp = torch.zeros(2, 1, device=DEV)
    ids, tp = torch.zeros(2, 3, dtype=torch.int32, device=DEV), torch.zeros(2, 3, device=DEV)
    ws = torch.zeros(c.logprob_workspace(2, 100), dtype=torch.uint8, device=DEV)
    good = dict(n=2, logits=x, tokens=tokens, logprob=lp, top_ids=ids, top_logprob=tp, workspace=ws)
    c.token_logprobs(**good)

    def refused(error, match, **kw):
        with pytest.raises(error, match=match):
            c.token_logprobs(**{**good, **kw})

    for scale in (0.0, -1.0, float("inf"), float("nan"), 2.0 ** 127):
        refused(KvrError, "scale must be finite", scale=scale)
    refused(ValueError, "logits: 2 rows", n=3)
    refused(ValueError, "dimensions", logits=x[0])
    refused(TypeError, "logits: expected", logits=x.double())
    refused(TypeError, "GPU tensor", logits=x.cpu())
    refused(TypeError, "tokens: expected int32", tokens=tokens.long())
    refused(ValueError, "tokens go with logprob", logprob=None)
    refused(ValueError, "top_ids with top_logprob", top_ids=None)
    refused(ValueError, "logprob: shape", logprob=lp[:1])
    refused(ValueError, "lse: shape", lse=torch.zeros(3, device=DEV))
    refused(KvrError, "the workspace has 0 bytes", workspace=None)
    refused(KvrError, "the workspace has", workspace=ws[:-16])
    refused(KvrError, r"top in \[0, 64\]", top_ids=torch.zeros(2, 65, dtype=torch.int32, device=DEV),
            top_logprob=torch.zeros(2, 65, device=DEV))
    refused(ValueError, "not contiguous", logprob=torch.zeros(2, 3, device=DEV)[:, :1])
    with pytest.raises(KvrError, match="vocab in"):
        c.logprob_workspace(2, 0)
    c.token_logprobs(0, x[:0], tokens[:0], lp[:0])
