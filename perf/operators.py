"""The row cache's operators: attention over resolved rows, row packing, and
the forking, freeing and compaction of the pages the rows live in.

Each case is one pass through one operator, either in plain torch operations
(`own` false) or through the package's entry points (`own` true).

  attend   attention of each request's new tokens over the rows its location
           vector (or its gathered buffer) names.  A row holds one latent per
           token: its key is the latent and a rope part, its value the latent.
  pack     RMS norm of new latents and their rows in the cache's format
           (bf16, or 8-bit codes with a scale for each 128 values).
  fork     the destinations' old state is freed and each becomes a copy of its
           source request that shares its ready pages; optionally some shared
           pages are then copied into pages of the destination's own.
  compact  live pages of a pool with holes move into its lowest pages.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 128      # values per scale of an 8-bit row
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.bfloat16}
PLACE_PAGE, PLACE_HOT = 1, 2
LOC_INVALID = -1  # 0xFFFFFFFF as int32


def row_bytes(fmt, d_v, d_rope):
    """Bytes of one row: the latent (2 bytes a value, or 1 and its scales,
    which take whole 16-byte pieces), then the rope part in 16 bits."""
    if fmt == "fp8":
        return d_v + -(-(d_v // GROUP) * 4 // 16) * 16 + 2 * d_rope
    return 2 * (d_v + d_rope)


def listed():
    return [
        # one request's decode step: the single-request workload's selection
        dict(name="attend one request", op="attend", n=1, nq=1, heads=16, k=256, fmt="bf16",
             d_v=512, d_rope=64, source="loc", union=0, ragged=False),
        # eight requests with all their heads: the shared-indices workload, one layer
        dict(name="attend shared indices", op="attend", n=8, nq=1, heads=64, k=2048, fmt="bf16",
             d_v=512, d_rope=64, source="loc", union=0, ragged=False),
        # 64 requests, few heads each (heads split over devices): 8-bit rows
        dict(name="attend few heads", op="attend", n=64, nq=1, heads=16, k=2048, fmt="fp8",
             d_v=512, d_rope=64, source="loc", union=0, ragged=False),
        # the long-context workload's decode step with every head on one device
        dict(name="attend long context", op="attend", n=64, nq=1, heads=128, k=2048, fmt="fp8",
             d_v=512, d_rope=64, source="loc", union=0, ragged=False),
        # a verification block: each of four queries reads its own rows of the union
        dict(name="attend verify block", op="attend", n=32, nq=4, heads=16, k=2048, fmt="bf16",
             d_v=512, d_rope=64, source="loc", union=3277, ragged=False),
        # ragged counts (none, one, all), odd heads, half precision, gathered rows
        dict(name="attend ragged", op="attend", n=37, nq=3, heads=23, k=1001, fmt="f16",
             d_v=256, d_rope=64, source="rows", union=0, ragged=True),
        # one decoded token for each of 64 requests
        dict(name="pack decode", op="pack", rows=64, fmt="fp8", src="bf16", d_v=512, d_rope=64),
        # the import of a 32768-row history for four layers
        dict(name="pack import", op="pack", rows=131072, fmt="fp8", src="bf16", d_v=512,
             d_rope=64),
        # one request forks another: the single-request workload's sizes
        dict(name="fork one", op="fork", pairs=1, layers=1, H=4096, R=1152, P=64, T=128, B=512,
             ready=0.5, decoded=5, copies=0),
        # four requests fork into four, some pages copied
        dict(name="fork four", op="fork", pairs=4, layers=2, H=8192, R=1152, P=64, T=256, B=4096,
             ready=0.7, decoded=33, copies=32),
        # a small pool after a few requests left
        dict(name="compact small pool", op="compact", requests=4, pages=256, R=1152, P=64,
             layers=1, holes=0.3),
        # a large pool of short rows after a third of it was freed
        dict(name="compact large pool", op="compact", requests=64, pages=16384, R=656, P=64,
             layers=1, holes=0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "pack", "fork", "compact"])
    if op == "attend":
        fmt = rng.choice(["bf16", "f16", "fp8"])
        d_v, d_rope = rng.choice([(512, 64), (512, 64), (512, 0), (256, 64), (256, 0)])
        while True:
            n, nq = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 5])
            heads, k = _log(rng, 1, 128), _log(rng, 1, 2048)
            if n * nq * heads * k <= 64 * 128 * 2048:
                break
        source = rng.choice(["loc", "loc", "rows"])
        union = rng.randint(k, min(8192, 2 * k + 7)) if nq > 1 and rng.random() < 0.5 else 0
        return dict(op=op, n=n, nq=nq, heads=heads, k=k, fmt=fmt, d_v=d_v, d_rope=d_rope,
                    source=source, union=union, ragged=rng.random() < 0.5)
    if op == "pack":
        d_v, d_rope = rng.choice([(512, 64), (512, 64), (512, 0), (256, 64)])
        return dict(op=op, rows=_log(rng, 1, 131072), fmt=rng.choice(["fp8", "fp8", "bf16", "f16"]),
                    src=rng.choice(["bf16", "bf16", "f16", "f32"]), d_v=d_v, d_rope=d_rope)
    if op == "fork":
        return dict(op=op, pairs=rng.randint(1, 4), layers=rng.randint(1, 2),
                    H=_log(rng, 300, 8192), R=rng.choice([656, 1152]), P=rng.choice([16, 48, 64]),
                    T=rng.choice([0, 37, 128, 256]), B=_log(rng, 64, 4096),
                    ready=round(rng.uniform(0, 1), 2), decoded=rng.randint(0, 40),
                    copies=rng.choice([0, 3]))
    return dict(op=op, requests=rng.randint(2, 64), pages=_log(rng, 64, 16384),
                R=rng.choice([656, 656, 1152]) if rng.random() < 0.5 else 656,
                P=rng.choice([16, 64]), layers=1, holes=round(rng.uniform(0.02, 0.5), 2))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1000003 * int(seed) + 17)


def _rand(g, hi, shape):
    return torch.randint(0, max(1, hi), shape, generator=g, device=DEV, dtype=torch.int64)


def _latents(g, n, d):
    """Latents after their norm: zero mean, unit size, a few larger channels."""
    x = torch.randn(n, d, generator=g, device=DEV)
    return x * (1 + 2 * (torch.arange(d, device=DEV) % 67 == 5))


def _rows_of(g, count, fmt, d_v, d_rope):
    """`count` rows of random latents in the cache's format, uint8 [count][R]."""
    out = torch.empty(count, row_bytes(fmt, d_v, d_rope), dtype=torch.uint8, device=DEV)
    for a in range(0, count, 1 << 17):
        b = min(count, a + (1 << 17))
        out[a:b] = _pack_plain(_latents(g, b - a, d_v), None, 0.0,
                               torch.randn(b - a, d_rope, generator=g, device=DEV), fmt)
    return out


def prepare(case, seed):
    return {"attend": _prepare_attend, "pack": _prepare_pack, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, _gen(seed))


def _prepare_attend(c, g):
    n, nq, heads, k, fmt = c["n"], c["nq"], c["heads"], c["k"], c["fmt"]
    d_v, d_rope = c["d_v"], c["d_rope"]
    stride = c["union"] or k
    R, P, T, B = row_bytes(fmt, d_v, d_rope), 64, 256, min(8192, max(64, stride))
    H = max(1024, 2 * k)
    pages = n * (H // P) // 2
    # tail, pool and hot cache in one allocation, as a serving process has them
    at = [0, n * T, n * T + pages * P, n * T + pages * P + n * B]
    arena = _rows_of(g, at[3], fmt, d_v, d_rope)
    req = torch.arange(n, device=DEV)[:, None]
    place = torch.rand(n, stride, generator=g, device=DEV)
    place = torch.where(place < 0.06, 0, torch.where(place < 0.5, PLACE_PAGE, PLACE_HOT))
    index = torch.where(place == 0, _rand(g, T, (n, stride)),
                        torch.where(place == PLACE_PAGE, _rand(g, pages * P, (n, stride)),
                                    torch.argsort(torch.rand(n, B, generator=g, device=DEV),
                                                  dim=1)[:, :stride] if stride <= B
                                    else _rand(g, B, (n, stride))))
    word = (place << 30) | index
    loc = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
    count = torch.full((n,), stride, dtype=torch.int32, device=DEV)
    if c["ragged"]:
        count = _rand(g, stride + 1, (n,)).to(torch.int32)
        count[0] = stride
        if n > 2:
            count[1:3] = torch.tensor([0, 1], device=DEV)
        loc = torch.where(torch.rand(n, stride, generator=g, device=DEV) < 0.03, LOC_INVALID, loc)
    s = dict(c, stride=stride, R=R, P=P, T=T, B=B, H=H, pages=pages, arena=arena, at=at, loc=loc,
             count=count, req=req, scale=1.0 / math.sqrt(d_v / 4 + d_rope), rows=None, map=None)
    if c["union"]:  # each query's own k distinct rows of the union
        s["map"] = torch.argsort(torch.rand(n, nq, stride, generator=g, device=DEV),
                                 dim=2)[:, :, :k].to(torch.int32).contiguous()
    if c["source"] == "rows":
        s["rows"] = arena[_rand(g, at[3], (n * stride,))].view(n, stride, R)
    typ = TYPES[fmt]
    s["q"] = torch.randn(n, nq, heads, d_v + d_rope, generator=g, device=DEV).to(typ)
    s["out"] = torch.empty(n, nq, heads, d_v, dtype=typ, device=DEV)
    s["lse"] = torch.empty(n, nq, heads, dtype=torch.float32, device=DEV)
    if own:
        s["ctx"] = _context(n, 1, H, 0, P, T, B, R, min(8192, stride), pages,
                            [arena[at[0]:at[1]]], [arena[at[1]:at[2]]], [arena[at[2]:]])
        s["workspace"] = torch.empty(
            s["ctx"].attend_workspace(n, nq, heads, d_v, k), dtype=torch.uint8, device=DEV)
    return s


def _prepare_pack(c, g):
    d_v, d_rope = c["d_v"], c["d_rope"]
    src = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[c["src"]]
    s = dict(c, R=row_bytes(c["fmt"], d_v, d_rope), eps=1e-6)
    # latents before their norm: token sizes differ
    size = torch.exp(torch.randn(c["rows"], 1, generator=g, device=DEV))
    s["latent"] = (_latents(g, c["rows"], d_v) * size).to(src)
    s["rope"] = torch.randn(c["rows"], d_rope, generator=g, device=DEV).to(src)
    s["weight"] = 1 + 0.1 * torch.randn(d_v, generator=g, device=DEV)
    s["packed"] = torch.empty(c["rows"], s["R"], dtype=torch.uint8, device=DEV)
    if own:
        s["ctx"] = _context(1, 1, 0, 1, 1, 0, 1, s["R"], 1, 0, [None], [None],
                            [torch.empty(s["R"], dtype=torch.uint8, device=DEV)])
    return s


def _prepare_fork(c, g):
    m, NL, H, R, P, T, B = (c[x] for x in ("pairs", "layers", "H", "R", "P", "T", "B"))
    n, npg, full, rows = 2 * m, -(-H // P), H // P, H + 64
    ready = int(round(c["ready"] * full))
    pages = max(1, m * ready + c["copies"])
    i32 = dict(dtype=torch.int32, device=DEV)
    s = dict(c, n=n, npg=npg, rows=rows, pages=pages,
             src=torch.arange(m, **i32), dst=torch.arange(m, n, **i32))
    phys = torch.randperm(pages, generator=g, device=DEV)
    pm = torch.full((m, npg), -1, dtype=torch.int64, device=DEV)
    if ready:
        at = torch.argsort(torch.rand(m, full, generator=g, device=DEV), dim=1)[:, :ready]
        pm.scatter_(1, at, phys[:m * ready].view(m, ready))
    s["page_map"] = torch.cat([pm, torch.full_like(pm, -1)]).to(torch.int32)
    s["host_valid"] = torch.cat([pm < 0, torch.zeros_like(pm, dtype=torch.bool)]).to(torch.uint8)
    s["L"] = torch.cat([H + _rand(g, c["decoded"] + 1, (m,)), torch.zeros(m, device=DEV)]).int()
    tags = torch.argsort(torch.rand(m, max(H, B), generator=g, device=DEV), dim=1)[:, :B]
    tags = torch.where(torch.rand(m, B, generator=g, device=DEV) < 0.8, tags, -1)
    s["tag"] = torch.cat([tags, torch.full_like(tags, -1)]).to(torch.int32)
    s["stamp"] = torch.cat([_rand(g, 1000, (m, B)) * (tags >= 0), torch.zeros_like(tags)]).int()
    s["clock"] = torch.cat([1000 + _rand(g, 9, (m,)), _rand(g, 1, (m,))]).to(torch.int32)
    byte = lambda *shape: torch.randint(0, 256, shape, generator=g, device=DEV,  # noqa: E731
                                        dtype=torch.uint8)
    s["tail"] = [byte(n, T, R) for _ in range(NL)]
    s["pool"] = [byte(pages, P, R) for _ in range(NL)]
    s["hot"] = [byte(n, B, R) for _ in range(NL)]
    s["host"] = []
    for _ in range(NL):
        h = torch.empty(n, rows, R, dtype=torch.uint8, pin_memory=True)
        h.copy_(byte(n, rows, R))
        s["host"].append(h)
    # physical pages no request maps, and the destinations' entries that get them
    nc = min(c["copies"], m * ready)
    s["spare"] = phys[m * ready:m * ready + nc].to(torch.int32)
    flat = torch.nonzero(pm.view(-1) >= 0).view(-1)
    flat = flat[torch.randperm(flat.numel(), generator=g, device=DEV)[:nc]]
    s["copy_req"] = (flat // npg + m).to(torch.int32)
    s["copy_page"] = (flat % npg).to(torch.int32)
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
    s["refs"][pm[pm >= 0]] = 1
    s["free"] = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
    s["free_count"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    s["status"] = torch.zeros(max(1, nc), dtype=torch.int32, device=DEV)
    if own:
        x = s["ctx"] = _context(n, NL, H, 64, P, T, B, R, min(B, 64), pages, s["tail"], s["pool"],
                                s["hot"], s["host"],
                                meta=[s[k] for k in ("L", "page_map", "host_valid", "tag",
                                                     "stamp", "clock")])
        x.bind_page_refs(s["refs"])
        s["workspace"] = torch.empty(x.pool_workspace(), dtype=torch.uint8, device=DEV)
    return s


def _prepare_compact(c, g):
    n, pages, R, P, NL = (c[x] for x in ("requests", "pages", "R", "P", "layers"))
    live = max(1, int(round((1 - c["holes"]) * pages)))
    npg = -(-live // n) + 3
    phys = torch.randperm(pages, generator=g, device=DEV)[:live]
    at = torch.randperm(n * npg, generator=g, device=DEV)[:live]
    pm = torch.full((n * npg,), -1, dtype=torch.int64, device=DEV)
    pm[at] = phys
    i32 = dict(dtype=torch.int32, device=DEV)
    refs = torch.zeros(pages, **i32)
    refs[phys] = 1
    s = dict(c, npg=npg, page_map0=pm.view(n, npg).to(torch.int32), refs0=refs,
             page_map=torch.empty(n, npg, **i32), refs=torch.empty(pages, **i32),
             moves=torch.full((pages, 2), -1, **i32), move_count=torch.zeros(1, **i32),
             pool=[torch.randint(0, 256, (pages, P, R), generator=g, device=DEV,
                                 dtype=torch.uint8) for _ in range(NL)])
    if own:
        H = npg * P
        s["host_valid"] = torch.zeros(n, npg, dtype=torch.uint8, device=DEV)
        byte = dict(dtype=torch.uint8, device=DEV)
        x = s["ctx"] = _context(n, NL, H, 0, P, 0, 1, R, 1, pages, [None] * NL, s["pool"],
                                [torch.empty(n, R, **byte) for _ in range(NL)],
                                meta=[torch.full((n,), H, **i32), s["page_map"], s["host_valid"],
                                      torch.full((n, 1), -1, **i32), torch.zeros(n, 1, **i32),
                                      torch.zeros(n, **i32)])
        x.bind_page_refs(s["refs"])
        s["workspace"] = torch.empty(x.pool_workspace(), dtype=torch.uint8, device=DEV)
    return s


def _context(n, NL, H, new, P, T, B, R, cap, pages, tail, pool, hot, host=None, meta=None):
    """A context of the package over the given buffers."""
    from hierarchical_sparse_kv_resolve_amd import Context
    x = Context(n_req=n, n_layers=NL, history_rows=H, max_new_rows=new, page_rows=P, tail_rows=T,
                hot_slots=B, row_bytes=R, sel_cap=cap, pool_pages=pages)
    if host is None:
        host = [torch.empty(n, H + new, R, dtype=torch.uint8, pin_memory=True)
                for _ in range(NL)]
    if meta is not None:
        x.bind_metadata(*meta)
    for l in range(NL):
        x.bind_layer(l, tail[l], pool[l], hot[l], host[l])
    x.buffers = (tail, pool, hot, host, meta)
    return x


# ------------------------------------------------------------------ passes

def run(state):
    op = state["op"]
    if own:
        return {"attend": _attend_own, "pack": _pack_own, "fork": _fork_own,
                "compact": _compact_own}[op](state)
    return {"attend": _attend, "pack": _pack, "fork": _fork, "compact": _compact}[op](state)


def _unpack(rows, fmt, d_v, d_rope):
    """Keys (latent, rope) of rows uint8 [..., R] in 32 bits."""
    if fmt != "fp8":
        return rows.view(TYPES[fmt]).float()
    n_s = d_v // GROUP
    sc = rows[..., d_v:d_v + 4 * n_s].contiguous().view(torch.float32)
    c = rows[..., :d_v].contiguous().view(torch.float8_e4m3fn).float()
    c = (c.view(*sc.shape, GROUP) * sc[..., None]).view(c.shape)
    r = rows[..., row_bytes(fmt, d_v, 0):].contiguous().view(torch.bfloat16).float()
    return torch.cat([c, r], dim=-1)


def _attend(s):
    n, nq, heads, k, d_v = s["n"], s["nq"], s["heads"], s["k"], s["d_v"]
    loc, stride = s["loc"], s["stride"]
    valid = (loc != LOC_INVALID) & (torch.arange(stride, device=DEV) < s["count"][:, None])
    if s["rows"] is None:
        place, index = (loc >> 30) & 3, (loc & 0x3FFFFFFF).long()
        index = torch.where(place == 0, s["req"] * s["T"] + index,
                            torch.where(place == PLACE_PAGE, s["at"][1] + index,
                                        s["at"][2] + s["req"] * s["B"] + index))
    else:
        index = torch.arange(n * stride, device=DEV).view(n, stride)
    if s["map"] is not None:
        pick = s["map"].view(n, nq * k).long()
        index, valid = index.gather(1, pick), valid.gather(1, pick)
    src = s["arena"] if s["rows"] is None else s["rows"].view(n * stride, -1)
    rows = src[torch.where(valid, index, 0)]
    key = _unpack(rows, s["fmt"], d_v, s["d_rope"]) * 1.0
    key = torch.where(valid[..., None], key, 0.0)
    q = s["q"].float() * s["scale"]
    if s["map"] is not None:
        key, valid = key.view(n, nq, k, -1), valid.view(n, nq, 1, k)
    else:
        key, valid = key[:, None], valid[:, None, None]
        q = q.view(n, 1, nq * heads, -1)
    score = torch.matmul(q, key.transpose(-1, -2).contiguous())
    score = torch.where(valid, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, key[..., :d_v].contiguous()) / torch.where(total == 0, 1.0, total)
    s["out"].copy_(out.view(n, nq, heads, d_v))
    s["lse"].copy_((top + torch.log(total)).view(n, nq, heads))
    return {"out": s["out"], "lse": s["lse"]}


def _attend_own(s):
    s["ctx"].attend_rows(0, s["n"], None, s["q"], s["out"], fmt=s["fmt"], d_v=s["d_v"],
                         d_rope=s["d_rope"], scale=s["scale"], stride=s["stride"], loc=s["loc"],
                         rows=s["rows"], count=s["count"], map_=s["map"], lse=s["lse"],
                         workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _pack_plain(x, weight, eps, rope, fmt):
    """Rows of latents x and rope parts, after the norm where there is a weight."""
    n, d_v = x.shape
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(1, keepdim=True) + eps) * weight
    if fmt != "fp8":
        return torch.cat([x, rope.float()], 1).to(TYPES[fmt]).view(torch.uint8)
    x = x.view(n, d_v // GROUP, GROUP)
    sc = x.abs().amax(2) / E4M3_MAX
    sc = torch.where(sc == 0, 1.0, sc)
    code = (x / sc[..., None]).to(torch.float8_e4m3fn).view(n, d_v).view(torch.uint8)
    gap = torch.zeros(n, row_bytes(fmt, d_v, 0) - d_v - 4 * sc.shape[1], dtype=torch.uint8,
                      device=x.device)
    return torch.cat([code, sc.contiguous().view(torch.uint8), gap,
                      rope.to(torch.bfloat16).contiguous().view(torch.uint8).view(n, -1)], 1)


def _packed_values(s):
    """The values the packed rows stand for: views of the parts of a row."""
    p, d_v = s["packed"], s["d_v"]
    if s["fmt"] != "fp8":
        return {"row": p.view(TYPES[s["fmt"]])}
    at = row_bytes("fp8", d_v, 0)
    return {"code": p[:, :d_v].view(torch.float8_e4m3fn),
            "scale": p.view(torch.float32)[:, d_v // 4:d_v // 4 + d_v // GROUP],
            "rope": p.view(torch.bfloat16)[:, at // 2:]}


def _pack(s):
    s["packed"].copy_(_pack_plain(s["latent"], s["weight"], s["eps"], s["rope"], s["fmt"]))
    return _packed_values(s)


def _pack_own(s):
    s["ctx"].pack_rows(s["rows"], s["latent"], s["rope"], s["packed"], fmt=s["fmt"],
                       d_v=s["d_v"], d_rope=s["d_rope"], weight=s["weight"], eps=s["eps"])
    return _packed_values(s)


def _fork_outputs(s):
    return {k: s[k] for k in ("L", "page_map", "host_valid", "tag", "stamp", "clock", "refs",
                              "free", "free_count", "tail", "pool", "hot", "host")}


def _fork(s):
    src, dst = s["src"].long(), s["dst"].long()
    H, P, npg, rows, pages = s["H"], s["P"], s["npg"], s["rows"], s["pages"]
    # free what the destinations hold
    old = s["page_map"][dst].reshape(-1).long()
    s["refs"].index_add_(0, old.clamp(min=0), -(old >= 0).int())
    for name, v in (("L", 0), ("page_map", -1), ("host_valid", 0), ("tag", -1), ("stamp", 0),
                    ("clock", 0)):
        s[name][dst] = v
    is_free = s["refs"] == 0
    order = torch.argsort(torch.where(is_free, 0, 1), stable=True)
    n_free = is_free.sum()
    s["free_count"].copy_(n_free.view(1))
    ids = torch.arange(pages, device=DEV)
    s["free"].copy_(torch.where(ids < n_free, order, s["free"]))
    # share the sources' ready pages, copy the rest of their state
    pm = s["page_map"][src]
    s["refs"].index_add_(0, pm.reshape(-1).clamp(min=0).long(), (pm >= 0).reshape(-1).int())
    hv = (s["host_valid"][src] != 0) & (pm < 0)
    s["page_map"][dst] = pm
    s["host_valid"][dst] = hv.to(torch.uint8)
    for name in ("L", "tag", "stamp", "clock"):
        s[name][dst] = s[name][src]
    filled = (s["tag"][src] >= 0)[..., None]
    pos = torch.arange(rows, device=DEV)
    has = torch.where(pos < H, hv[:, (pos // P).clamp(max=npg - 1)], pos < s["L"][src][:, None])
    for t, h, x in zip(s["tail"], s["hot"], s["host"]):
        t[dst] = t[src]
        h[dst] = torch.where(filled, h[src], h[dst])
        d = x.to(DEV, non_blocking=True)
        d[dst] = torch.where(has[..., None], d[src], d[dst])
        x.copy_(d, non_blocking=True)
    # shared pages copied into pages of the destinations' own
    r, p = s["copy_req"].long(), s["copy_page"].long()
    was, to = s["page_map"][r, p].long(), s["spare"].long()
    for x in s["pool"]:
        x[to] = x[was]
    s["refs"].index_add_(0, was, torch.full_like(was, -1, dtype=torch.int32))
    s["refs"][to] = 1
    s["page_map"][r, p] = s["spare"]
    return _fork_outputs(s)


def _fork_own(s):
    x, m = s["ctx"], s["pairs"]
    x.release_requests(m, s["dst"])
    x.list_free_pages(s["free"], s["free_count"], s["workspace"])
    x.fork_requests(m, s["src"], s["dst"])
    x.copy_pages(s["copy_req"].numel(), s["copy_req"], s["copy_page"], s["spare"], s["status"])
    return _fork_outputs(s)


def _compact(s):
    s["page_map"].copy_(s["page_map0"])
    s["refs"].copy_(s["refs0"])
    pages, refs, pm = s["pages"], s["refs"], s["page_map"]
    ids = torch.arange(pages, device=DEV)
    live = refs > 0
    n_live = live.sum()
    move = torch.nonzero(live & (ids >= n_live)).view(-1).flip(0)
    hole = torch.nonzero(~live & (ids < n_live)).view(-1)
    for x in s["pool"]:
        x[hole] = x[move]
    to = ids.clone()
    to[move] = hole
    pm.copy_(torch.where(pm >= 0, to[pm.clamp(min=0).long()], -1))
    refs[hole] = refs[move]
    refs[move] = 0
    k = hole.numel()
    s["moves"][:k] = torch.stack([move, hole], 1).int()
    s["move_count"].fill_(k)
    return _compact_outputs(s)


def _compact_own(s):
    s["page_map"].copy_(s["page_map0"])
    s["refs"].copy_(s["refs0"])
    s["ctx"].compact_pool(s["pages"], s["moves"], s["move_count"], s["workspace"])
    return _compact_outputs(s)


def _compact_outputs(s):
    return {k: s[k] for k in ("page_map", "refs", "moves", "move_count", "pool")}


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "attend":
        n, nq, heads, k, d_v, d_rope = (c[x] for x in ("n", "nq", "heads", "k", "d_v", "d_rope"))
        rows = c["union"] or k
        R = row_bytes(c["fmt"], d_v, d_rope)
        share = 0.5 if c["ragged"] else 1.0  # mean count of a ragged batch
        moved = n * rows * (R + 4) * share + 4 * n * nq * k * bool(c["union"])
        heads_all = n * nq * heads
        return {"bytes": moved + heads_all * (2 * (d_v + d_rope) + 2 * d_v + 4),
                "flops": 2 * heads_all * k * share * (2 * d_v + d_rope)}
    if c["op"] == "pack":
        d = c["d_v"] + c["d_rope"]
        e = 4 if c["src"] == "f32" else 2
        return {"bytes": c["rows"] * (d * e + row_bytes(c["fmt"], c["d_v"], c["d_rope"]))
                + 4 * c["d_v"], "flops": 8 * c["rows"] * c["d_v"]}
    if c["op"] == "fork":
        m, H, R, B = c["pairs"], c["H"], c["R"], c["B"]
        npg = -(-H // c["P"])
        host = H - int(round(c["ready"] * (H // c["P"]))) * c["P"] + c["decoded"] / 2
        rows = c["T"] + 0.8 * B + host
        return {"bytes": 2 * m * (c["layers"] * R * rows + 8 * B + 5 * npg)
                + 2 * c["copies"] * c["layers"] * c["P"] * R, "flops": 0}
    moved = c["pages"] * c["holes"] * (1 - c["holes"])
    return {"bytes": 2 * moved * c["P"] * c["R"] * c["layers"] + 16 * c["pages"], "flops": 0}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    if case["op"] == "attend":
        return _attend_exact(_prepare_attend(case, _gen(seed)))
    if case["op"] == "pack":
        return _pack_exact(_prepare_pack(case, _gen(seed)))
    return None  # whole numbers only


def _attend_exact(s):
    """softmax over each request's list of rows, one request and query at a time."""
    n, nq, heads, d_v, fmt = s["n"], s["nq"], s["heads"], s["d_v"], s["fmt"]
    out = torch.zeros(n, nq, heads, d_v, dtype=torch.float64, device=DEV)
    lse = torch.full((n, nq, heads), -math.inf, dtype=torch.float64, device=DEV)
    base = {0: lambda i: i * s["T"], 1: lambda i: s["at"][1], 2: lambda i: s["at"][2] + i * s["B"]}
    counts = s["count"].tolist()
    for i in range(n):
        words = s["loc"][i].long() & 0xFFFFFFFF
        if s["rows"] is not None:
            raw = s["rows"][i]
        else:
            off = torch.zeros_like(words)
            for place in range(3):
                off[words >> 30 == place] = base[place](i)
            raw = s["arena"][torch.where(words == 0xFFFFFFFF, 0, off + (words & 0x3FFFFFFF))]
        if fmt == "fp8":
            code = raw[:, :d_v].contiguous().view(torch.float8_e4m3fn).double()
            sc = raw[:, d_v:d_v + d_v // 32].contiguous().view(torch.float32).double()
            val = code * torch.repeat_interleave(sc, GROUP, dim=1)
            rope = raw[:, raw.shape[1] - 2 * s["d_rope"]:].contiguous().view(torch.bfloat16)
            key = torch.cat([val, rope.double()], 1)
        else:
            key = raw.view(TYPES[fmt]).double()
        for a in range(nq):
            pick = torch.arange(s["stride"], device=DEV) if s["map"] is None else s["map"][i, a].long()
            pick = pick[(words[pick] != 0xFFFFFFFF) & (pick < counts[i])]
            if pick.numel() == 0:
                continue
            kk = key[pick]
            x = (s["q"][i, a].double() @ kk.T) * s["scale"]
            lse[i, a] = torch.logsumexp(x, 1)
            out[i, a] = torch.exp(x - lse[i, a][:, None]) @ kk[:, :d_v]
    return {"out": out, "lse": lse}


def _pack_exact(s):
    x = s["latent"].double()
    x = x / torch.sqrt((x * x).sum(1, keepdim=True) / s["d_v"] + s["eps"]) * s["weight"].double()
    rope = s["rope"].double()
    if s["fmt"] != "fp8":
        return {"row": torch.cat([x, rope], 1)}
    top = torch.stack([t.abs().max(1).values for t in x.split(GROUP, dim=1)], 1)
    scale = torch.where(top > 0, top / E4M3_MAX, 1.0)
    return {"code": x / torch.repeat_interleave(scale, GROUP, dim=1), "scale": scale, "rope": rope}
