"""A drafter's steps and their verification as a program runs them: rotary positions
of queries and keys, keys and values into the window, attention over it, lengths
advanced, tokens scored, what is rejected dropped.  Every quantity is followed in
64 bits from the values the step before left on the device, so that each stage's
error is its own (the bounds of the stages are derived in their own tests; here
they are the coarse ones of the types)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import draft_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Drafter:
    """Two layers of random weights over the package's calls."""

    def __init__(self, n, W, C, heads, kv, d, vocab, layers=2, seed=0):
        from hierarchical_sparse_kv_resolve_amd import Context, DraftRing, rope_frequencies
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.n, self.heads, self.kv, self.d, self.layers, self.vocab = n, heads, kv, d, layers, vocab
        self.codes = torch.full((layers, n, C // 64, kv, 2, 64 * d), 0x7F, dtype=torch.uint8,
                                device=DEV)
        self.scales = torch.full((layers, n, C // 64, kv, 2), 255, dtype=torch.uint8, device=DEV)
        self.length = torch.zeros(n, dtype=torch.int32, device=DEV)
        self.high = torch.zeros(n, dtype=torch.int32, device=DEV)
        self.ring = DraftRing(n, W, C, 0, None, self.length, self.high)
        self.ring.bind_kv(layers, kv, d, self.codes, self.scales)
        self.ctx = Context(n_req=n, n_layers=1, history_rows=0, max_new_rows=1, page_rows=1,
                           tail_rows=0, hot_slots=1, row_bytes=16, sel_cap=1, pool_pages=0)
        f, self.magnitude = rope_frequencies(d // 2, scaling="ramp", factor=8.0,
                                             original_length=256)
        self.freq = torch.from_numpy(f).to(DEV)
        width = heads * d
        rand = lambda *s: torch.randn(s, generator=g, device=DEV) * s[-2] ** -0.5  # noqa: E731
        self.embed = torch.randn(vocab, width, generator=g, device=DEV)
        self.w_in = [rand(width, (heads + 2 * kv) * d).bfloat16() for _ in range(layers)]
        self.w_out = [rand(width, width).bfloat16() for _ in range(layers)]
        self.w_head = rand(width, vocab).bfloat16()
        self.seen = []  # what each layer's stages took and gave

    def step(self, tokens, count=None, mask="causal"):
        """tokens int32 [n, rows] at the positions after the rows kept: logits of them."""
        n, rows = tokens.shape
        ws = torch.empty(max(1, self.ring.attend_workspace(n, rows, self.heads)),
                         dtype=torch.uint8, device=DEV)
        x = self.embed[tokens.long()]
        pos = (self.length[:, None] + torch.arange(rows, device=DEV)).int().reshape(-1)
        self.seen = []
        for l in range(self.layers):
            proj = (x.bfloat16().view(n * rows, -1) @ self.w_in[l]).view(n * rows, -1, self.d)
            q, k = proj[:, :self.heads], proj[:, self.heads:self.heads + self.kv]
            v = proj[:, self.heads + self.kv:].view(n, rows, self.kv, self.d)
            before = proj.clone()
            # half of each head is rotated, in place, queries and keys in one call
            self.ctx.rotate_rows(n * rows, pos, self.freq, q, key=k, d_rot=self.d // 2,
                                 layout="half", at=self.d // 4, key_at=self.d // 4,
                                 magnitude=self.magnitude)
            kk = k.view(n, rows, self.kv, self.d) if k.is_contiguous() else \
                k.unflatten(0, (n, rows))
            self.ring.write_kv(l, n, None, kk, v, count)
            out = torch.zeros(n, rows, self.heads, self.d, dtype=torch.bfloat16, device=DEV)
            lse = torch.zeros(n, rows, self.heads, device=DEV)
            self.ring.attend(l, n, None, q.unflatten(0, (n, rows)), out, scale=self.d ** -0.5,
                             mask=mask, count=count, lse=lse, workspace=ws)
            self.seen.append((before, pos, proj.clone(), out, lse, self.codes[l].clone(),
                              self.scales[l].clone()))
            x = x + out.view(n, rows, -1).float() @ self.w_out[l].float()
        self.ring.advance(n, None, rows, count)
        return (x.bfloat16().view(n * rows, -1) @ self.w_head).view(n, rows, -1)

    def score(self, logits, tokens, top=5):
        n, rows, vocab = logits.shape
        flat = logits.reshape(n * rows, vocab)
        lp = torch.zeros(n * rows, 1, device=DEV)
        ids = torch.zeros(n * rows, top, dtype=torch.int32, device=DEV)
        tp = torch.zeros(n * rows, top, device=DEV)
        ent = torch.zeros(n * rows, device=DEV)
        ws = torch.empty(self.ctx.logprob_workspace(n * rows, vocab), dtype=torch.uint8, device=DEV)
        self.ctx.token_logprobs(n * rows, flat, tokens.reshape(-1, 1).contiguous(), lp,
                                entropy=ent, top_ids=ids, top_logprob=tp, workspace=ws)
        return lp.view(n, rows), ids.view(n, rows, top), tp.view(n, rows, top), ent.view(n, rows)


def check_stages(D, lengths, mirrors, rows, count, mask="causal"):
    """Each layer's stages against 64 bits, from what the stage before left."""
    n, d, kv, heads = D.n, D.d, D.kv, D.heads
    a, half = d // 4, d // 4
    for l, (before, pos, after, out, lse, codes, scales) in enumerate(D.seen):
        # rotation
        turns = pos.double()[:, None].cpu() * D.freq.cpu()
        ang = 2 * np.pi * (turns - torch.round(turns))
        c, s = (D.magnitude * f(ang)[:, None] for f in (torch.cos, torch.sin))
        x, y = before.double().cpu(), after.double().cpu()
        turned = slice(0, heads + kv)
        u, v = x[:, turned, a:a + half], x[:, turned, a + half:a + 2 * half]
        for got, want in ((y[:, turned, a:a + half], u * c - v * s),
                          (y[:, turned, a + half:a + 2 * half], v * c + u * s)):
            # half a bf16 step, and 32-bit factors
            assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * (u.abs() + v.abs())
                    + 2.0 ** -120).all()
        x[:, turned, a:a + 2 * half] = y[:, turned, a:a + 2 * half]
        assert torch.equal(x, y)
        # the window, bit for bit
        proj = y.view(n, rows, heads + 2 * kv, d).numpy()
        w = mirrors[l]
        for r in range(n):
            m = rows if count is None else count[r]
            assert w.length[r] == lengths[r]
            w.write(r, proj[r, :m, heads:heads + kv], proj[r, :m, heads + kv:])
        want_codes, want_scales = w.device_layout()
        got_codes, got_scales = codes.cpu().numpy(), scales.cpu().numpy()
        used = got_scales != 255
        assert np.array_equal(got_scales[used], want_scales[used])
        touched = used[..., None] & np.ones(got_codes.shape, dtype=bool)
        assert np.array_equal(got_codes[touched], want_codes[touched])
        # attention
        o64, l64 = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for r in range(n):
            m = rows if count is None else count[r]
            for j in range(m):
                lo, hi = ref.span(mask, lengths[r], m, j, w.W)
                keys, vals = w.rows(r, lo, hi)
                for h in range(kv):
                    at = slice(h * (heads // kv), (h + 1) * (heads // kv))
                    o, s, spread, size = ref.attend(proj[r, j, at], keys[h], vals[h], d ** -0.5)
                    assert (np.abs(l64[r, j, at] - s) <= 2.0 ** -14 * (1 + size)).all()
                    tol = (2.0 ** -8 + 2.0 ** -12 * (1 + size))[:, None] * spread + 2.0 ** -8 * np.abs(o)
                    assert (np.abs(o64[r, j, at] - o) <= tol).all()
            w.advance(r, m)


@pytest.mark.parametrize("heads,kv,d,W", [(4, 2, 64, 100), (6, 1, 128, 70)])
def test_drafting_and_verification(heads, kv, d, W):
    """A prompt, then rounds of drafting three tokens, verifying them as a block of
    other tokens' scores, and dropping what is rejected."""
    n, vocab, C = 3, 1000, 256
    D = Drafter(n, W, C, heads, kv, d, vocab)
    mirrors = [ref.Window(n, W, C, kv, d) for _ in range(D.layers)]
    rng = np.random.default_rng(0)
    token = lambda *s: torch.from_numpy(rng.integers(0, vocab, s).astype(np.int32)).to(DEV)  # noqa: E731

    def run(tokens, count=None, mask="causal"):
        lengths = D.length.tolist()
        c = None if count is None else torch.tensor(count, dtype=torch.int32, device=DEV)
        logits = D.step(tokens, c, mask)
        check_stages(D, lengths, mirrors, tokens.shape[1], count, mask)
        return logits

    run(token(n, 80), [80, 13, 1])
    for round_ in range(6):
        drafted, last = [], token(n, 1)
        for _ in range(3):
            logits = run(last)
            lp, ids, tp, ent = D.score(logits, last)
            x = torch.log_softmax(logits.double(), -1)
            assert torch.equal(ids[..., 0].long(), logits.float().argmax(-1))
            assert ((tp - x.gather(-1, ids.long())).abs() <= 1e-5 * (1 + tp.abs())).all()
            assert ((ent + (x.exp() * x).sum(-1)).abs() <= 1e-4).all()
            last = ids[..., 0].contiguous()
            drafted.append(last)
        # scores of the drafted tokens under (other) logits of a verification block
        block = torch.cat(drafted, 1)
        target = torch.randn(n, 3, vocab, device=DEV).bfloat16()
        lp, *_ = D.score(target, block)
        want = torch.log_softmax(target.double(), -1).gather(-1, block.long()[..., None])[..., 0]
        assert ((lp - want).abs() <= 1e-5 * (1 + want.abs())).all()
        accept = [int(a) for a in rng.integers(0, 4, n)]
        length = D.length.tolist()
        keep = [length[r] - 3 + accept[r] for r in range(n)]
        status = torch.full((n,), 9, dtype=torch.int32, device=DEV)
        D.ring.rollback(n, None, torch.tensor(keep, dtype=torch.int32, device=DEV), status)
        assert (status == 0).all()
        for w in mirrors:
            w.length[:] = keep
    # a block of tokens that see one another
    run(token(n, 5), [5, 2, 4], "block")


def test_layers_read_back():
    """What the steps left in each layer, read back, is what its mirror holds."""
    D = Drafter(2, 64, 128, 2, 1, 64, 300, seed=1)
    mirrors = [ref.Window(2, 64, 128, 1, 64) for _ in range(D.layers)]
    for rows in (40, 1, 1, 33):
        tokens = torch.randint(0, 300, (2, rows), dtype=torch.int32, device=DEV)
        lengths = D.length.tolist()
        D.step(tokens)
        check_stages(D, lengths, mirrors, rows, None)
    for l, w in enumerate(mirrors):
        k = torch.zeros(2, 64, 1, 64, device=DEV)
        v = torch.zeros_like(k)
        vis = torch.zeros(2, dtype=torch.int32, device=DEV)
        D.ring.read_kv(l, 2, None, k, v, vis)
        assert vis.tolist() == [64, 64]
        for r in range(2):
            keys, vals = w.rows(r, 75 - 64, 75)
            assert np.array_equal(k[r].cpu().double().numpy(), keys.transpose(1, 0, 2))
            assert np.array_equal(v[r].cpu().double().numpy(), vals.transpose(1, 0, 2))
