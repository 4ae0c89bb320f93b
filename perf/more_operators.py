"""The operators of a drafter's step and of the scoring of what it drafted.

Each case is one pass through one operator, either in plain torch operations
(`own` false) or through the package's entry points (`own` true).

  rotate   rotary positions of queries and keys: pairs of a head's rotated part
           turned by position times frequency, the rest of the head passed on.
  write    new tokens' keys and values into the drafter's window: e4m3 codes,
           one power-of-two scale for each block of 64 tokens and head.
  read     the visible window back in 16 or 32 bits, oldest row first.
  attend   attention of new tokens' queries over the window, sliding and causal,
           over their whole block, or over the kept rows only.
  logprob  log probabilities of given tokens, the entropy and the most likely
           alternatives of each row of logits.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 64         # tokens that share a scale
E4M3_MAX = 448.0
MIN_EXP = -100     # smallest exponent of a scale
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one decoded token of 64 requests: the rope part of latent queries and
        # of the shared key, positions in a long context
        dict(name="rotate decode", op="rotate", n=64, heads=16, d_head=576, at=512, d_rot=64,
             kv_heads=1, kd_head=64, kat=0, layout="interleaved", typ="bf16", far=524288),
        # a 32768-token prompt: whole heads, halves
        dict(name="rotate prompt", op="rotate", n=32768, heads=16, d_head=128, at=0, d_rot=128,
             kv_heads=4, kd_head=128, kat=0, layout="half", typ="bf16", far=32768),
        # one token for each of 64 requests
        dict(name="write decode", op="write", n=64, rows=1, kv_heads=8, d=128, window=1024,
             capacity=1152, typ="bf16", ragged=False, first=0.0, dropped=0),
        # prompts of eight requests in chunks of 4096 tokens
        dict(name="write prompt", op="write", n=8, rows=4096, kv_heads=8, d=128, window=4096,
             capacity=8256, typ="bf16", ragged=False, first=0.0, dropped=0),
        # one request's window for a check or another layout
        dict(name="read one", op="read", n=1, kv_heads=8, d=128, window=1024, capacity=1152,
             typ="bf16", first=0.0),
        # the windows of 32 requests
        dict(name="read windows", op="read", n=32, kv_heads=8, d=128, window=4096, capacity=4224,
             typ="bf16", first=0.0),
        # one request drafts a token
        dict(name="attend one", op="attend", n=1, nq=1, heads=32, kv_heads=8, d=128, window=1024,
             capacity=1152, mask="causal", ragged=False, first=0.0),
        # 64 requests draft a token each over long windows
        dict(name="attend decode", op="attend", n=64, nq=1, heads=32, kv_heads=8, d=128,
             window=4096, capacity=4224, mask="causal", ragged=False, first=0.0),
        # the accepted tokens of 32 requests, none to four each, small heads; some
        # requests are still short
        dict(name="attend accepted", op="attend", n=32, nq=4, heads=14, kv_heads=2, d=64,
             window=2000, capacity=2112, mask="causal", ragged=True, first=0.3),
        # a chunk of a prompt
        dict(name="attend prompt", op="attend", n=1, nq=2048, heads=32, kv_heads=8, d=128,
             window=4096, capacity=8192, mask="causal", ragged=False, first=0.0),
        # one drafted token and its alternatives
        dict(name="logprob one", op="logprob", n=1, vocab=131072, m=1, top=20, typ="bf16",
             banned=0.0),
        # a verification block: four tokens of 32 requests
        dict(name="logprob verify", op="logprob", n=128, vocab=131072, m=1, top=20, typ="bf16",
             banned=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "write", "read", "attend", "attend", "logprob"])
    if op == "rotate":
        d_rot = rng.choice([16, 32, 64, 64, 96, 128])
        d_head = rng.choice([d_rot, d_rot, 128 if d_rot <= 128 else d_rot, 576])
        heads, kv = _log(rng, 1, 64), rng.choice([1, 1, 4])
        n = min(_log(rng, 1, 32768), 32768 * 20 * 128 // ((heads + kv) * d_head))
        return dict(op=op, n=n, heads=heads, d_head=d_head, at=rng.choice([0, d_head - d_rot]),
                    d_rot=d_rot, kv_heads=kv, kd_head=d_rot, kat=0,
                    layout=rng.choice(["interleaved", "half"]),
                    typ=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    far=_log(rng, 1000, 1 << 20))
    d, kv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 3, 4, 8])
    window = _log(rng, 64, 4096)
    if op == "write":
        while True:
            n, rows = _log(rng, 1, 64), _log(rng, 1, 4096)
            if n * rows * kv * d <= 8 * 4096 * 8 * 128:
                break
        capacity = -(-(window + rows + 70) // BLOCK) * BLOCK
        return dict(op=op, n=n, rows=rows, kv_heads=kv, d=d, window=window, capacity=capacity,
                    typ=rng.choice(["bf16", "bf16", "f16", "f32"]), ragged=rng.random() < 0.5,
                    first=rng.choice([0.0, 0.4]), dropped=rng.choice([0, 0, 5]))
    if op == "read":
        n = max(1, min(_log(rng, 1, 32), 32 * 4096 * 8 * 128 // (window * kv * d)))
        return dict(op=op, n=n, kv_heads=kv, d=d, window=window,
                    capacity=-(-(window + 5) // BLOCK) * BLOCK,
                    typ=rng.choice(["bf16", "bf16", "f16", "f32"]), first=rng.choice([0.0, 0.4]))
    if op == "attend":
        group = rng.choice([1, 2, 4, 5, 7, 8, 16])
        if rng.random() < 0.7:
            n, nq = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 5])
        else:
            n, nq = rng.randint(1, 3), _log(rng, 16, 2048)
        while n * nq * group * kv * window * d > 2048 * 32 * 4096 * 128:
            n, nq = max(1, n // 2), max(1, nq // 2)
        return dict(op=op, n=n, nq=nq, heads=group * kv, kv_heads=kv, d=d, window=window,
                    capacity=-(-(window + nq + 63) // BLOCK) * BLOCK,
                    mask=rng.choice(["causal", "causal", "block", "kept"]),
                    ragged=rng.random() < 0.5, first=rng.choice([0.0, 0.4]))
    vocab = _log(rng, 1000, 131072)
    return dict(op=op, n=min(_log(rng, 1, 512), 128 * 131072 // vocab), vocab=vocab,
                m=rng.choice([0, 1, 1, 1, 5]), top=rng.choice([0, 1, 5, 20, 64]),
                typ=rng.choice(["bf16", "bf16", "f16", "f32"]), banned=rng.choice([0.0, 0.0, 0.9]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1000003 * int(seed) + 29)


def _rand(g, hi, shape):
    return torch.randint(0, max(1, hi), shape, generator=g, device=DEV, dtype=torch.int64)


def _randn(g, shape, typ=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(typ)


def prepare(case, seed):
    g = _gen(seed)
    s = {"rotate": _prepare_rotate, "write": _prepare_write, "read": _prepare_read,
         "attend": _prepare_attend, "logprob": _prepare_logprob}[case["op"]](case, g)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program of the package keeps for its calls."""
    from hierarchical_sparse_kv_resolve_amd import Context, DraftRing
    if s["op"] in ("rotate", "logprob"):
        s["ctx"] = Context(n_req=1, n_layers=1, history_rows=0, max_new_rows=1, page_rows=1,
                           tail_rows=0, hot_slots=1, row_bytes=16, sel_cap=1, pool_pages=0)
        if s["op"] == "logprob":
            s["workspace"] = torch.empty(s["ctx"].logprob_workspace(s["n"], s["vocab"]),
                                         dtype=torch.uint8, device=DEV)
        return
    s["ring"] = DraftRing(s["n"], s["window"], s["capacity"], 0, None, s["length"], s["high"])
    s["ring"].bind_kv(1, s["kv_heads"], s["d"], s["codes"], s["scales"])
    if s["op"] == "attend":
        s["workspace"] = torch.empty(s["ring"].attend_workspace(s["n"], s["nq"], s["heads"]),
                                     dtype=torch.uint8, device=DEV)


def _prepare_rotate(c, g):
    n, typ = c["n"], TYPES[c["typ"]]
    # frequencies in turns per position, the slow ones stretched for long contexts
    i = torch.arange(c["d_rot"] // 2, device=DEV, dtype=torch.float64)
    f = 10000.0 ** (-2 * i / c["d_rot"]) / (2 * math.pi)
    keep = ((f * 4096 - 1) / 31).clamp(0, 1)
    s = dict(c, frequencies=f * keep + f / 16 * (1 - keep), magnitude=1.0 + 0.1 * math.log(16.0),
             positions=_rand(g, c["far"], (n,)).to(torch.int32),
             q=_randn(g, (n, c["heads"], c["d_head"]), typ),
             k=_randn(g, (n, c["kv_heads"], c["kd_head"]), typ))
    s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    return s


def _window(c, g, extra):
    """A drafter's window in use: lengths, codes and scales of one layer.  `first`: the
    share of requests that have not filled their ring once."""
    n, C, d, kv = c["n"], c["capacity"], c["d"], c["kv_heads"]
    length = C + _rand(g, 3 * C, (n,))
    short = torch.rand(n, generator=g, device=DEV) < c["first"]
    length = torch.where(short, _rand(g, max(1, C - extra), (n,)), length)
    nb = C // BLOCK
    size = torch.exp2(_rand(g, 4, (1, n, nb, kv, 2)) - 7).float()
    scales = (torch.log2(size) + 127).to(torch.uint8)
    codes = torch.empty(1, n, nb, kv, 2, BLOCK * d, dtype=torch.uint8, device=DEV)
    x = codes.view(-1)
    for a in range(0, x.numel(), 1 << 26):
        part = x[a:a + (1 << 26)]
        part.copy_((_randn(g, part.shape) * 80).clamp(-E4M3_MAX, E4M3_MAX)
                   .to(torch.float8_e4m3fn).view(torch.uint8))
    return dict(c, length=length.to(torch.int32), high=length.to(torch.int32), codes=codes,
                scales=scales)


def _counts(c, g, rows):
    if not c["ragged"]:
        return None
    count = _rand(g, rows + 1, (c["n"],))
    count[0] = rows
    return count.to(torch.int32)


def _prepare_write(c, g):
    s = _window(c, g, c["rows"])
    # dropped by an earlier verification: written past the kept length
    s["high"] = s["high"] + c["dropped"]
    shape = (c["n"], c["rows"], c["kv_heads"], c["d"])
    # one projection's output; a few larger channels and tokens of different sizes
    both = torch.empty(shape[0], shape[1], 2, *shape[2:], dtype=TYPES[c["typ"]], device=DEV)
    both.copy_(_randn(g, both.shape) * (1 + 5 * (torch.arange(c["d"], device=DEV) % 37 == 3))
               * torch.exp(0.5 * _randn(g, (shape[0], shape[1], 1, 1, 1))))
    s["k"], s["v"] = both[:, :, 0], both[:, :, 1]
    s["count"] = _counts(c, g, c["rows"])
    return s


def _prepare_read(c, g):
    s = _window(c, g, 0)
    shape = (c["n"], c["window"], c["kv_heads"], c["d"])
    s["k"] = torch.zeros(shape, dtype=TYPES[c["typ"]], device=DEV)
    s["v"] = torch.zeros(shape, dtype=TYPES[c["typ"]], device=DEV)
    s["visible"] = torch.zeros(c["n"], dtype=torch.int32, device=DEV)
    return s


def _prepare_attend(c, g):
    s = _window(c, g, c["nq"])
    shape = (c["n"], c["nq"], c["heads"], c["d"])
    s["q"] = _randn(g, shape, torch.bfloat16)
    s["out"] = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros(shape[:3], dtype=torch.float32, device=DEV)
    s["count"] = _counts(c, g, c["nq"])
    s["scale"] = 1.0 / math.sqrt(c["d"])
    return s


def _prepare_logprob(c, g):
    n, vocab, m, top = (c[x] for x in ("n", "vocab", "m", "top"))
    # a few likely tokens over a wide floor
    logits = _randn(g, (n, vocab)) * 2
    logits.scatter_add_(1, _rand(g, vocab, (n, 40)), 6 + 3 * _randn(g, (n, 40)))
    if c["banned"]:
        logits[torch.rand(n, vocab, generator=g, device=DEV) < c["banned"]] = -math.inf
    f32 = dict(dtype=torch.float32, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(c, logits=logits.to(TYPES[c["typ"]]), scale=1.0 / 0.8,
                tokens=_rand(g, vocab, (n, m)).to(torch.int32), logprob=torch.empty(n, m, **f32),
                lse=torch.empty(n, **f32), entropy=torch.empty(n, **f32),
                top_ids=torch.empty(n, top, **i32), top_logprob=torch.empty(n, top, **f32))


# ------------------------------------------------------------------ passes

def run(state):
    op = state["op"]
    if own:
        return {"rotate": _rotate_own, "write": _write_own, "read": _read_own,
                "attend": _attend_own, "logprob": _logprob_own}[op](state)
    return {"rotate": _rotate, "write": _write, "read": _read, "attend": _attend,
            "logprob": _logprob}[op](state)


def _turn(x, cos, sin, at, d, layout):
    """x [n, heads, d_head] with its pairs in [at, at + d) turned."""
    y, part = x.clone(), x[..., at:at + d].float()
    if layout == "half":
        a, b = part[..., :d // 2], part[..., d // 2:]
        part = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    y[..., at:at + d] = part.to(x.dtype)
    return y


def _rotate(s):
    turns = s["positions"].double()[:, None] * s["frequencies"]
    angle = (turns - torch.round(turns)) * (2 * math.pi)
    cos = (torch.cos(angle) * s["magnitude"]).float()[:, None]
    sin = (torch.sin(angle) * s["magnitude"]).float()[:, None]
    return {"q": _turn(s["q"], cos, sin, s["at"], s["d_rot"], s["layout"]),
            "k": _turn(s["k"], cos, sin, s["kat"], s["d_rot"], s["layout"])}


def _rotate_own(s):
    s["ctx"].rotate_rows(s["n"], s["positions"], s["frequencies"], s["q"], s["q_out"], s["k"],
                         s["k_out"], d_rot=s["d_rot"], layout=s["layout"], at=s["at"],
                         key_at=s["kat"], magnitude=s["magnitude"])
    return {"q": s["q_out"], "k": s["k_out"]}


def _scale(b):
    return torch.exp2(b.float() - 127)


def _dequantised(codes, scales, d):
    """Keys and values [..., kv, BLOCK, d] in 32 bits of blocks [..., kv, 2, BLOCK * d]."""
    x = codes.view(torch.float8_e4m3fn).float() * _scale(scales)[..., None]
    k = x[..., 0, :].unflatten(-1, (BLOCK, d))
    v = x[..., 1, :].unflatten(-1, (d, BLOCK)).transpose(-1, -2)
    return k, v


def _spread(x, p):
    """x [n, rows, ...] at the row numbers p [n, nb, BLOCK] (rows outside: any)."""
    n, rows = x.shape[:2]
    idx = p.clamp(0, rows - 1).view(n, -1)
    return x[torch.arange(n, device=DEV)[:, None], idx].view(*p.shape, *x.shape[2:])


def _write(s):
    n, rows, kv, d, C = s["n"], s["rows"], s["kv_heads"], s["d"], s["capacity"]
    nb = min((rows + BLOCK - 2) // BLOCK + 1, C // BLOCK)
    length, high = s["length"].long(), s["high"].long()
    count = s["count"].long() if s["count"] is not None else torch.full_like(length, rows)
    # the positions that the touched blocks' slots stand for on this lap
    first = length // BLOCK * BLOCK
    pos = (first[:, None, None] + torch.arange(nb, device=DEV)[:, None] * BLOCK
           + torch.arange(BLOCK, device=DEV))
    new = (pos >= length[:, None, None]) & (pos < (length + count)[:, None, None])
    # what a slot held before: the last position written there
    was = torch.where(pos < high[:, None, None], pos, pos - C)
    live = ~new & (was >= 0) & (was < length[:, None, None])
    req = torch.arange(n, device=DEV)[:, None]
    at = (pos[..., 0] // BLOCK) % (C // BLOCK)
    old_codes, old_scales = s["codes"][0][req, at], s["scales"][0][req, at]
    k, v = _dequantised(old_codes, old_scales, d)
    p = pos - length[:, None, None]
    nk, nv = _spread(s["k"], p).float(), _spread(s["v"], p).float()  # [n, nb, BLOCK, kv, d]
    # a token with a value that is not finite shows in its whole key
    bad = ~(torch.isfinite(nk).all(-1) & torch.isfinite(nv).all(-1))
    nk = torch.where(bad[..., None], math.nan, nk)
    nv = torch.where(torch.isfinite(nv), nv, 0.0)
    mask = lambda m: m[:, :, None, :, None]  # noqa: E731
    k = torch.where(mask(new), nk.transpose(2, 3), torch.where(mask(live), k, 0.0))
    v = torch.where(mask(new), nv.transpose(2, 3), torch.where(mask(live), v, 0.0))
    x = torch.stack([k.flatten(-2), v.transpose(-1, -2).flatten(-2)], 3)  # [n, nb, kv, 2, ...]
    top = torch.where(torch.isnan(x), 0.0, x.abs()).amax(-1)
    # smallest e with top <= 448 * 2^e: the quotient's exponent, or the next one
    e = torch.where(top > 0, torch.frexp(top / E4M3_MAX).exponent - 1, MIN_EXP)
    e = e.clamp(min=MIN_EXP)
    e = torch.where(top > E4M3_MAX * torch.exp2(e.float()), e + 1, e)
    codes = (x * torch.exp2(-e.float())[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    touched = new.any(-1)[..., None, None]
    s["codes"][0][req, at] = torch.where(touched[..., None], codes, old_codes)
    s["scales"][0][req, at] = torch.where(touched, (e + 127).to(torch.uint8), old_scales)
    return _cache(s)


def _cache(s):
    """The values that the cache's bytes stand for."""
    return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": _scale(s["scales"])}


def _write_own(s):
    s["ring"].write_kv(0, s["n"], None, s["k"], s["v"], count=s["count"])
    return _cache(s)


def _rows_at(s, pos):
    """Keys and values [n, rows, kv, d] in 32 bits of positions pos [n, rows]."""
    n, rows = pos.shape
    slot = pos % s["capacity"]
    req, blk, off = torch.arange(n, device=DEV)[:, None], slot // BLOCK, slot % BLOCK
    codes, sc = s["codes"][0], _scale(s["scales"][0][req, blk])  # [n, rows, kv, 2]
    kc = codes[..., 0, :].unflatten(-1, (BLOCK, s["d"])).transpose(2, 3)
    vc = codes[..., 1, :].unflatten(-1, (s["d"], BLOCK)).permute(0, 1, 4, 2, 3)
    k = kc[req, blk, off].view(torch.float8_e4m3fn).float() * sc[..., 0:1]
    v = vc[req, blk, off].view(torch.float8_e4m3fn).float() * sc[..., 1:2]
    return k, v


def _read(s):
    W, length = s["window"], s["length"].long()
    vis = length.clamp(max=W)
    row = torch.arange(W, device=DEV)
    seen = (row < vis[:, None])[..., None, None]
    k, v = _rows_at(s, (length - vis)[:, None] + row)
    s["k"].copy_(torch.where(seen, k.to(s["k"].dtype), s["k"]))
    s["v"].copy_(torch.where(seen, v.to(s["v"].dtype), s["v"]))
    s["visible"].copy_(vis)
    return {"k": s["k"], "v": s["v"], "visible": s["visible"]}


def _read_own(s):
    s["ring"].read_kv(0, s["n"], None, s["k"], s["v"], visible=s["visible"])
    return {"k": s["k"], "v": s["v"], "visible": s["visible"]}


def _attend(s):
    n, nq, heads, kv, d, W = (s[x] for x in ("n", "nq", "heads", "kv_heads", "d", "window"))
    length = s["length"].long()
    count = s["count"].long() if s["count"] is not None else torch.full_like(length, nq)
    j = torch.arange(nq, device=DEV)
    hi = {"causal": length[:, None] + j + 1, "block": (length + count)[:, None].expand(n, nq),
          "kept": length[:, None].expand(n, nq)}[s["mask"]]
    lo = (hi - W).clamp(min=0)
    first = lo.amin(1)
    pos = first[:, None] + torch.arange(W + (nq - 1 if s["mask"] == "causal" else 0), device=DEV)
    k, v = _rows_at(s, pos)
    k, v = k.transpose(1, 2), v.transpose(1, 2).contiguous()  # [n, kv, rows, d]
    q = s["q"].float().view(n, nq, kv, heads // kv, d).permute(0, 2, 1, 3, 4)
    q = q.reshape(n, kv, nq * (heads // kv), d) * s["scale"]
    score = torch.matmul(q, k.transpose(-1, -2).contiguous()).view(n, kv, nq, heads // kv, -1)
    p = pos[:, None, None, None]
    sees = (p >= lo[:, None, :, None, None]) & (p < hi[:, None, :, None, None])
    score = torch.where(sees, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w.flatten(2, 3), v).view(n, kv, nq, heads // kv, d)
    out = out / torch.where(total == 0, 1.0, total)
    out = out.permute(0, 2, 1, 3, 4).reshape(n, nq, heads, d)
    lse = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(n, nq, heads)
    given = (j < count[:, None])[..., None]
    s["out"].copy_(torch.where(given[..., None], out.to(torch.bfloat16), s["out"]))
    s["lse"].copy_(torch.where(given, lse, s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def _attend_own(s):
    s["ring"].attend(0, s["n"], None, s["q"], s["out"], scale=s["scale"], mask=s["mask"],
                     count=s["count"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _logprob(s):
    x = s["logits"].float()
    t = x * s["scale"]
    top = t.amax(1, keepdim=True)
    shifted = t - top
    e = torch.exp(shifted)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    logp = shifted - log_total
    s["logprob"].copy_(logp.gather(1, s["tokens"].long()))
    s["lse"].copy_((top + log_total)[:, 0])
    s["entropy"].copy_((log_total - torch.where(e > 0, e * shifted, 0.0).sum(1, keepdim=True)
                        / total)[:, 0])
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :s["top"]]
    got = logp.gather(1, ids)
    s["top_ids"].copy_(torch.where(got == -math.inf, -1, ids))
    s["top_logprob"].copy_(got)
    return _logprob_outputs(s)


def _logprob_outputs(s):
    return {k: s[k] for k in ("logprob", "lse", "entropy", "top_ids", "top_logprob")}


def _logprob_own(s):
    s["ctx"].token_logprobs(s["n"], s["logits"], s["tokens"], s["logprob"], lse=s["lse"],
                            entropy=s["entropy"], top_ids=s["top_ids"],
                            top_logprob=s["top_logprob"], scale=s["scale"],
                            workspace=s["workspace"])
    return _logprob_outputs(s)


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "rotate":
        e = 4 if c["typ"] == "f32" else 2
        values = c["n"] * (c["heads"] * c["d_head"] + c["kv_heads"] * c["kd_head"])
        turned = c["n"] * (c["heads"] + c["kv_heads"]) * c["d_rot"]
        return {"bytes": 2 * e * values + 4 * c["n"], "flops": 3 * turned}
    if c["op"] == "logprob":
        e, values = 4 if c["typ"] == "f32" else 2, c["n"] * c["vocab"]
        return {"bytes": e * values + c["n"] * (8 * c["m"] + 8 + 8 * c["top"]),
                "flops": 4 * values}
    d, kv = c["d"], c["kv_heads"]
    if c["op"] == "write":
        e = 4 if c["typ"] == "f32" else 2
        values = 2 * c["n"] * c["rows"] * kv * d * (0.5 if c["ragged"] else 1.0)
        return {"bytes": (e + 1) * values, "flops": 2 * values}
    if c["op"] == "read":
        e = 4 if c["typ"] == "f32" else 2
        values = 2 * c["n"] * c["window"] * kv * d * (1 - 0.5 * c["first"])
        return {"bytes": (e + 1) * values, "flops": values}
    share = (1 - 0.5 * c["first"]) * (0.5 if c["ragged"] else 1.0)
    queries = c["n"] * c["nq"] * c["heads"]
    rows = c["window"] + (c["nq"] - 1 if c["mask"] == "causal" else 0)
    return {"bytes": 2 * c["n"] * rows * kv * d * (1 - 0.5 * c["first"])
            + queries * (4 * d + 4) * (0.5 if c["ragged"] else 1.0),
            "flops": 4 * queries * c["window"] * d * share}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    g = _gen(seed)
    return {"rotate": lambda: _rotate_exact(_prepare_rotate(case, g)),
            "write": lambda: _write_exact(_prepare_write(case, g)),
            "read": lambda: _read_exact(_prepare_read(case, g)),
            "attend": lambda: _attend_exact(_prepare_attend(case, g)),
            "logprob": lambda: _logprob_exact(_prepare_logprob(case, g))}[case["op"]]()


def _rotate_exact(s):
    """Each pair as a complex number times magnitude * exp(i angle)."""
    turns = s["positions"].double()[:, None] * s["frequencies"]
    factor = torch.polar(torch.full_like(turns, s["magnitude"]), 2 * math.pi * (turns % 1.0))

    def one(x, at):
        x, d = x.double(), s["d_rot"]
        part = x[..., at:at + d]
        half = s["layout"] == "half"
        pair = part.unflatten(-1, (2, d // 2)).transpose(-1, -2) if half else \
            part.unflatten(-1, (d // 2, 2))
        turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * factor[:, None])
        x[..., at:at + d] = (turned.transpose(-1, -2) if half else turned).flatten(-2)
        return x

    return {"q": one(s["q"], s["at"]), "k": one(s["k"], s["kat"])}


def _write_exact(s):
    """One request and block of its new tokens at a time."""
    n, d, C = s["n"], s["d"], s["capacity"]
    codes = s["codes"].view(torch.float8_e4m3fn).double()
    scales = torch.pow(2.0, s["scales"].double() - 127)
    length, high = s["length"].tolist(), s["high"].tolist()
    count = [s["rows"]] * n if s["count"] is None else s["count"].tolist()
    for i in range(n):
        a, end = length[i], length[i] + count[i]
        holds = [p for p in range(max(0, high[i] - C), a)]  # rows kept so far
        holds = {p % C for p in holds}
        while a < end:
            stop = min(end, (a // BLOCK + 1) * BLOCK)
            blk, off = a % C // BLOCK, a % BLOCK
            c, sc = codes[0, i, blk], scales[0, i, blk]  # [kv, 2, BLOCK * d], [kv, 2]
            x = c * sc[..., None]
            k, v = x[:, 0].view(-1, BLOCK, d).clone(), x[:, 1].view(-1, d, BLOCK).clone()
            dead = [t for t in range(BLOCK) if blk * BLOCK + t not in holds]
            k[:, dead], v[:, :, dead] = 0.0, 0.0
            src = slice(a - length[i], stop - length[i])
            k[:, off:off + stop - a] = s["k"][i, src].double().transpose(0, 1)
            v[:, :, off:off + stop - a] = s["v"][i, src].double().permute(1, 2, 0)
            both = torch.stack([k.flatten(1), v.flatten(1)], 1)
            e = torch.ceil(torch.log2(both.abs().amax(-1) / E4M3_MAX)).clamp(min=MIN_EXP)
            scales[0, i, blk] = torch.pow(2.0, e)
            codes[0, i, blk] = both / torch.pow(2.0, e)[..., None]
            a = stop
    return {"codes": codes, "scales": scales}


def _row_exact(s, i):
    """A request's ring in 64 bits: keys and values [kv, capacity, d]."""
    d, kv = s["d"], s["kv_heads"]
    x = s["codes"][0, i].view(torch.float8_e4m3fn).double()
    x = x * torch.pow(2.0, s["scales"][0, i].double() - 127)[..., None]
    k = x[:, :, 0].view(-1, kv, BLOCK, d).transpose(0, 1).reshape(kv, -1, d)
    v = x[:, :, 1].view(-1, kv, d, BLOCK).permute(1, 0, 3, 2).reshape(kv, -1, d)
    return k, v


def _read_exact(s):
    ks, vs = s["k"].double(), s["v"].double()
    length = s["length"].tolist()
    for i in range(s["n"]):
        k, v = _row_exact(s, i)
        vis = min(length[i], s["window"])
        at = torch.arange(length[i] - vis, length[i], device=DEV) % s["capacity"]
        ks[i, :vis], vs[i, :vis] = k[:, at].transpose(0, 1), v[:, at].transpose(0, 1)
    return {"k": ks, "v": vs, "visible": None}


def _attend_exact(s):
    """softmax over each query's rows, one request and kv head at a time."""
    n, nq, kv, d = s["n"], s["nq"], s["kv_heads"], s["d"]
    group = s["heads"] // kv
    out, lse = s["out"].double(), s["lse"].double()
    length = s["length"].tolist()
    count = [nq] * n if s["count"] is None else s["count"].tolist()
    for i in range(n):
        keys, values = _row_exact(s, i)
        m = count[i]
        if m == 0:
            continue
        last = {"causal": length[i] + m, "block": length[i] + m, "kept": length[i]}[s["mask"]]
        start = max(0, last - s["window"] - (m - 1 if s["mask"] == "causal" else 0))
        pos = torch.arange(start, last, device=DEV)
        end = torch.full((m,), last, device=DEV) if s["mask"] != "causal" else \
            length[i] + 1 + torch.arange(m, device=DEV)
        hide = (pos[None] >= end[:, None]) | (pos[None] < (end - s["window"])[:, None])
        for h in range(kv):
            kk, vv = keys[h, pos % s["capacity"]], values[h, pos % s["capacity"]]
            q = s["q"][i, :m, h * group:(h + 1) * group].double().flatten(0, 1)
            x = (q @ kk.T).view(m, group, -1) * s["scale"]
            x = x.masked_fill(hide[:, None], -math.inf).flatten(0, 1)
            ls = torch.logsumexp(x, 1) if pos.numel() else x.new_full((m * group,), -math.inf)
            p = torch.where(ls[:, None] == -math.inf, 0.0, torch.exp(x - ls[:, None]))
            out[i, :m, h * group:(h + 1) * group] = (p @ vv).view(m, group, d)
            lse[i, :m, h * group:(h + 1) * group] = ls.view(m, group)
    return {"out": out, "lse": lse}


def _logprob_exact(s):
    logp = torch.log_softmax(s["logits"].double() * s["scale"], 1)
    p = torch.exp(logp)
    order = torch.argsort(s["logits"], dim=1, descending=True, stable=True)[:, :s["top"]]
    return {"logprob": logp.gather(1, s["tokens"].long()),
            "lse": torch.logsumexp(s["logits"].double() * s["scale"], 1),
            "entropy": -torch.where(p > 0, p * logp, 0.0).sum(1), "top_ids": None,
            "top_logprob": logp.gather(1, order)}
