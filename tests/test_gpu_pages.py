"""Forking and freeing requests, copying, listing and compacting pages against
plain models of the same state changes, and a run of packing, resolving,
forking, compaction and attention together."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import attend_reference as ref

pytestmark = pytest.mark.gpu

POISON = 0x5A


class State:
    """A source with random metadata and payload, its device copy, and the
    plain forms of the page operators on the host copy."""

    META = ("L", "page_map", "host_valid", "tag", "stamp", "clock")
    PAYLOAD = ("tail", "pool", "hot", "host")

    def __init__(self, seed, *, n_req=6, H=330, P=16, T=21, B=40, R=48, NL=2, new=9, ready=0.5,
                 spare=11, users=None):
        from hierarchical_sparse_kv_resolve_amd import Context
        rng = np.random.default_rng(seed)
        self.rng, self.n_req, self.H, self.P, self.T, self.B, self.R = rng, n_req, H, P, T, B, R
        self.NL, self.new = NL, new
        npg, full = -(-H // P), H // P
        self.npg, self.full = npg, full
        users = n_req if users is None else users  # requests that hold something
        want = rng.random((users, full)) < ready
        self.pages = int(want.sum()) + spare
        phys = rng.permutation(self.pages)
        self.page_map = np.full((n_req, npg), -1, np.int32)
        sub = self.page_map[:users, :full]
        sub[want] = phys[:want.sum()]
        self.host_valid = np.zeros((n_req, npg), np.uint8)
        self.host_valid[:users] = (self.page_map[:users] < 0) | (rng.random((users, npg)) < 0.2)
        self.L = np.zeros(n_req, np.int32)
        self.L[:users] = H + rng.integers(0, new + 1, users)
        self.tag = np.full((n_req, B), -1, np.int32)
        self.stamp = np.zeros((n_req, B), np.int32)
        for r in range(users):
            fill = rng.random(B) < 0.7
            self.tag[r, fill] = rng.choice(H + B, int(fill.sum()), replace=False)
            self.stamp[r, fill] = rng.integers(1, 50, int(fill.sum()))
        self.clock = np.where(np.arange(n_req) < users, 50, 0).astype(np.int32)
        byte = lambda *s: rng.integers(0, 256, s, dtype=np.uint8)  # noqa: E731
        self.tail = [byte(n_req, T, R) for _ in range(NL)]
        self.pool = [byte(self.pages, P, R) for _ in range(NL)]
        self.hot = [byte(n_req, B, R) for _ in range(NL)]
        self.host = [byte(n_req, H + new, R) for _ in range(NL)]
        self.refs = np.bincount(self.page_map[self.page_map >= 0],
                                minlength=self.pages).astype(np.int32)
        self.ctx = Context(n_req=n_req, n_layers=NL, history_rows=H, max_new_rows=new, page_rows=P,
                           tail_rows=T, hot_slots=B, row_bytes=R, sel_cap=32,
                           pool_pages=self.pages)
        self.dev = {k: torch.from_numpy(getattr(self, k).copy()).cuda() for k in self.META}
        for k in ("tail", "pool", "hot"):
            self.dev[k] = [torch.from_numpy(x.copy()).cuda() for x in getattr(self, k)]
        self.dev["host"] = [torch.from_numpy(x.copy()).pin_memory() for x in self.host]
        self.dev["refs"] = torch.full((self.pages,), 99, dtype=torch.int32, device="cuda")
        self.ctx.bind_metadata(*[self.dev[k] for k in self.META])
        for l in range(NL):
            self.ctx.bind_layer(l, *[self.dev[k][l] if self.dev[k][l].numel() else None
                                     for k in self.PAYLOAD])
        self.ctx.bind_page_refs(self.dev["refs"])
        self.ctx.count_page_refs()
        self.ws = torch.empty(self.ctx.pool_workspace(), dtype=torch.uint8, device="cuda")

    def check(self):
        torch.cuda.synchronize()
        for k in self.META + ("refs",):
            assert np.array_equal(self.dev[k].cpu().numpy(), getattr(self, k)), k
        for k in self.PAYLOAD:
            for l in range(self.NL):
                assert np.array_equal(self.dev[k][l].cpu().numpy(), getattr(self, k)[l]), (k, l)

    # plain forms
    def release(self, r):
        for p in range(self.npg):
            if self.page_map[r, p] >= 0:
                self.refs[self.page_map[r, p]] -= 1
        self.page_map[r], self.host_valid[r], self.tag[r], self.stamp[r] = -1, 0, -1, 0
        self.L[r] = self.clock[r] = 0

    def fork(self, s, d):
        self.release(d)
        self.L[d], self.clock[d] = self.L[s], self.clock[s]
        self.tag[d], self.stamp[d], self.page_map[d] = self.tag[s], self.stamp[s], self.page_map[s]
        for p in range(self.npg):
            if self.page_map[s, p] >= 0:
                self.refs[self.page_map[s, p]] += 1
            elif self.host_valid[s, p]:
                self.host_valid[d, p] = 1
        for l in range(self.NL):
            self.tail[l][d] = self.tail[l][s]
            for b in range(self.B):
                if self.tag[s, b] >= 0:
                    self.hot[l][d, b] = self.hot[l][s, b]
            for pos in range(self.L[s]):
                if pos >= self.H or self.host_valid[d, pos // self.P]:
                    self.host[l][d, pos] = self.host[l][s, pos]

    def compact(self, most):
        moves = []
        live = int((self.refs > 0).sum())
        high = [p for p in range(self.pages - 1, live - 1, -1) if self.refs[p] > 0]
        low = [p for p in range(live) if self.refs[p] <= 0]
        for a, b in list(zip(high, low))[:most]:
            moves.append((a, b))
            self.page_map[self.page_map == a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
            for l in range(self.NL):
                self.pool[l][b] = self.pool[l][a]
        return moves


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("seed,kw", [
    (1, {}), (2, dict(R=1152, P=64, H=400)), (3, dict(R=656, NL=3, ready=1.0)),
    (4, dict(T=0, H=16, P=16)), (5, dict(H=15, P=16, spare=0)), (6, dict(new=0, ready=0.0, spare=0)),
    (7, dict(H=0, T=5, spare=2)), (8, dict(B=300, T=200, H=130, P=7))])
def test_fork(seed, kw):
    """Forks of one request twice, of another once; then again over them."""
    s = State(seed, **kw)
    s.check()
    for pairs in ([(0, 4), (0, 5), (2, 1)], [(4, 2), (1, 0)], [(5, 5)], [(3, 4)]):
        status = torch.full((len(pairs),), 77, dtype=torch.int32, device="cuda")
        s.ctx.fork_requests(len(pairs), ints(*[a for a, _ in pairs]), ints(*[b for _, b in pairs]),
                            status)
        good = [a != b for a, b in pairs]
        for (a, b), ok in zip(pairs, good):
            if ok:
                s.fork(a, b)
        s.check()
        assert status.cpu().tolist() == [0 if ok else -1 for ok in good]


def test_fork_bad_entries():
    """Ids out of range, a destination named twice, a request on both sides: each
    changes nothing, the other entries take place."""
    s = State(11)
    src, dst = [0, 6, 1, 0, 2, 3, -1], [1, 2, 5, 4, 4, 7, 2]
    status = torch.full((7,), 77, dtype=torch.int32, device="cuda")
    # n is at most n_req = 6
    from hierarchical_sparse_kv_resolve_amd import KvrError
    with pytest.raises(KvrError, match="request count 7"):
        s.ctx.fork_requests(7, ints(*src), ints(*dst), status)
    s.ctx.fork_requests(6, ints(*src[:6]), ints(*dst[:6]), status)
    s.fork(0, 4)
    s.check()
    assert status.cpu().tolist() == [-1, -1, -1, 0, -1, -1, 77]
    s.ctx.fork_requests(0, None, None)
    with pytest.raises(KvrError, match="src_ids and dst_ids"):
        s.ctx.fork_requests(1, None, ints(1))
    s.check()


def test_release():
    s = State(12)
    s.ctx.fork_requests(1, ints(0), ints(3))
    s.fork(0, 3)
    status = torch.full((4,), 77, dtype=torch.int32, device="cuda")
    s.ctx.release_requests(4, ints(0, 5, 0, 6), status)
    s.release(0)
    s.release(5)
    s.check()
    assert status.cpu().tolist() == [0, 0, -1, -1]
    s.ctx.release_requests(2, ints(0, 3))
    s.release(3)
    s.check()


def test_reclaim_and_restore_with_counts():
    """A shared page stays in use until its last entry lets it go; a restore
    into a page in use is refused, into a free one counts it."""
    s = State(13, ready=0.6)
    s.ctx.fork_requests(1, ints(0), ints(1))
    s.fork(0, 1)
    p = int(np.nonzero(s.page_map[0] >= 0)[0][0])
    ph = int(s.page_map[0, p])
    freed = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    status = torch.full((1,), 77, dtype=torch.int32, device="cuda")

    def reclaim(r):
        s.ctx.reclaim_pages(1, ints(r), ints(p), freed, status)
        if not s.host_valid[r, p]:
            for l in range(s.NL):
                s.host[l][r, p * s.P:(p + 1) * s.P] = s.pool[l][ph]
        s.host_valid[r, p], s.page_map[r, p] = 1, -1
        s.refs[ph] -= 1
        s.check()
        assert freed.item() == ph and status.item() == 0

    reclaim(0)
    assert s.refs[ph] == 1
    s.ctx.restore_pages(1, ints(0), ints(p), ints(ph), status)
    s.check()
    assert status.item() == -6  # KVR_E_STATE: request 1 still reads it
    reclaim(1)
    assert s.refs[ph] == 0
    s.ctx.restore_pages(1, ints(0), ints(p), ints(ph), status)
    s.page_map[0, p], s.refs[ph] = ph, 1
    for l in range(s.NL):
        s.pool[l][ph] = s.host[l][0, p * s.P:(p + 1) * s.P]
    s.check()
    assert status.item() == 0


def test_shared_page_reclaimed_by_all_in_one_call():
    """Every entry of a shared page lets it go in one call: each gets its own host
    copy, each names the page, and it is free."""
    s = State(63, ready=0.6)
    s.ctx.fork_requests(2, ints(0, 0), ints(1, 4))
    s.fork(0, 1)
    s.fork(0, 4)
    p = int(np.nonzero(s.page_map[0] >= 0)[0][0])
    ph = int(s.page_map[0, p])
    assert s.refs[ph] == 3
    freed = torch.full((4,), 77, dtype=torch.int32, device="cuda")
    status = torch.full((4,), 77, dtype=torch.int32, device="cuda")
    s.ctx.reclaim_pages(4, ints(1, 0, 4, 0), ints(p, p, p, p), freed, status)
    for r in (0, 1, 4):
        if not s.host_valid[r, p]:
            for l in range(s.NL):
                s.host[l][r, p * s.P:(p + 1) * s.P] = s.pool[l][ph]
        s.host_valid[r, p], s.page_map[r, p] = 1, -1
    s.refs[ph] = 0
    s.check()
    assert freed.cpu().tolist() == [ph, ph, ph, -1] and status.cpu().tolist() == [0] * 4


def test_copy_pages():
    """Shared pages become the entries' own; bad entries change nothing."""
    s = State(14, ready=0.6)
    s.ctx.fork_requests(2, ints(0, 0), ints(3, 4))
    s.fork(0, 3)
    s.fork(0, 4)
    free = np.nonzero(s.refs == 0)[0]
    held = np.nonzero(s.page_map[3] >= 0)[0]
    away = int(np.nonzero(s.page_map[3, :s.full] < 0)[0][0])
    assert len(free) >= 4 and len(held) >= 3
    rows = [(3, held[0], free[0], 0), (4, held[0], free[1], 0), (3, held[0], free[2], -1),
            (3, held[1], free[0], -1), (3, away, free[2], -6), (6, 0, free[2], -1),
            (3, s.full, free[3], -1), (3, held[1], s.page_map[0, held[1]], -6),
            (3, held[2], s.pages, -2), (0, held[1], free[-1], 0)]
    # an earlier entry's page or physical page counts, whatever became of it
    seen_pg, seen_ph = set(), set()
    for i, (r, p, ph, st) in enumerate(rows):
        if (r, p) in seen_pg or ph in seen_ph:
            rows[i] = (r, p, ph, -1)
        seen_pg.add((r, p))
        seen_ph.add(ph)
    status = torch.full((len(rows),), 77, dtype=torch.int32, device="cuda")
    s.ctx.copy_pages(len(rows), ints(*[int(x[0]) for x in rows]), ints(*[int(x[1]) for x in rows]),
                     ints(*[int(x[2]) for x in rows]), status)
    for r, p, ph, st in rows:
        if st == 0:
            old = s.page_map[r, p]
            for l in range(s.NL):
                s.pool[l][ph] = s.pool[l][old]
            s.refs[old] -= 1
            s.refs[ph] += 1
            s.page_map[r, p] = ph
    s.check()
    assert status.cpu().tolist() == [x[3] for x in rows]


@pytest.mark.parametrize("seed,kw", [
    (21, {}), (22, dict(H=9000, P=4, R=16, NL=1, B=8, n_req=8, ready=0.7)),
    (23, dict(ready=0.0, spare=5)), (24, dict(ready=1.0, spare=0)), (25, dict(ready=0.0, spare=0)),
    (26, dict(H=40000, P=2, R=16, NL=1, B=8, n_req=7, new=0, T=0, ready=0.9, spare=3000))])
def test_free_list_and_compaction(seed, kw):
    """Free lists and compaction before and after requests leave, with shared
    pages, with a bound on the moves and without."""
    s = State(seed, **kw)
    s.ctx.fork_requests(1, ints(0), ints(2))
    s.fork(0, 2)
    for step in range(4):
        free = torch.full((max(1, s.pages),), -7, dtype=torch.int32, device="cuda")
        count = torch.full((1,), -7, dtype=torch.int32, device="cuda")
        s.ctx.list_free_pages(free, count, s.ws)
        want = np.nonzero(s.refs == 0)[0]
        torch.cuda.synchronize()
        assert count.item() == len(want)
        got = free.cpu().numpy()
        assert np.array_equal(got[:len(want)], want) and (got[len(want):] == -7).all()
        most = (5, 0, s.pages, 1 << 30)[step]
        moves = torch.full((min(most, s.pages) + 1, 2), -7, dtype=torch.int32, device="cuda")
        n = torch.full((1,), -7, dtype=torch.int32, device="cuda")
        s.ctx.compact_pool(most, moves, n, s.ws)
        plan = s.compact(most)
        s.check()
        assert n.item() == len(plan)
        got = moves.cpu().numpy()
        assert np.array_equal(got[:len(plan)], np.array(plan, np.int32).reshape(-1, 2))
        assert (got[len(plan):] == -7).all()
        if step == 1:  # request 0's pages are still shared by 2
            s.ctx.release_requests(2, ints(0, 1))
            s.release(0)
            s.release(1)


@pytest.mark.parametrize("seed", [61, 62])
def test_fork_before_the_fills_have_run(seed):
    """A fork between a resolve and its fills (of several layers): the copy's hot
    slots hold their rows' bytes in every layer, whether the fills run later
    (into the source's slots) or not, and so do those of a copy of the copy,
    also where a page became ready meanwhile; the copy's next resolve hits them."""
    s = State(seed, n_req=4, users=1, NL=3, R=48, H=330, P=16, T=21, B=60, new=9, ready=0.4)
    # one truth: every place holds the row's own bytes
    byte = s.rng.integers(0, 256, (s.NL, s.H + s.new, s.R), dtype=np.uint8)
    L = int(s.L[0])
    for l in range(s.NL):
        for p in range(s.npg):
            lo, hi = p * s.P, min(s.H, p * s.P + s.P)
            if s.page_map[0, p] >= 0:
                s.dev["pool"][l][int(s.page_map[0, p]), :hi - lo] = torch.from_numpy(byte[l, lo:hi]).cuda()
            if s.host_valid[0, p]:
                s.dev["host"][l][0, lo:hi] = torch.from_numpy(byte[l, lo:hi])
        s.dev["host"][l][0, s.H:L] = torch.from_numpy(byte[l, s.H:L])
        for pos in range(max(0, L - s.T), L):
            s.dev["tail"][l][0, pos % s.T] = torch.from_numpy(byte[l, pos]).cuda()
        s.dev["hot"][l][0] = POISON
    s.dev["tag"].fill_(-1)
    s.dev["stamp"].zero_()
    k, i32 = 32, dict(dtype=torch.int32, device="cuda")

    def resolve(r, sel):
        out = dict(loc=torch.full((1, k), -1, **i32), fills=torch.zeros(1, s.B, 2, **i32),
                   count=torch.zeros(1, **i32), status=torch.full((1,), 77, **i32))
        s.ctx.resolve_rows(1, ints(r), torch.from_numpy(sel.astype(np.int32)[None]).cuda(), None, k,
                           out["loc"], out["fills"], out["count"], -1, out["status"])
        torch.cuda.synchronize()
        assert out["status"].item() == 0
        return out

    def fill(r, got):
        s.ctx.reuse_locations(1, list(range(s.NL)), 1, ints(r), got["loc"], None, None, k,
                              got["fills"], got["count"])

    def slots(r):
        """Every tagged slot of request r holds its row, in each layer."""
        torch.cuda.synchronize()
        tag = s.dev["tag"][r].cpu().numpy()
        assert (tag >= 0).any()
        for l in range(s.NL):
            hot = s.dev["hot"][l][r].cpu().numpy()
            assert np.array_equal(hot[tag >= 0], byte[l][tag[tag >= 0]]), (r, l)

    def rows(r, sel, got):
        out = [torch.zeros(1, k, s.R, dtype=torch.uint8, device="cuda") for _ in range(s.NL)]
        s.ctx.gather_rows(list(range(s.NL)), 1, ints(r), got["loc"], None, k, out)
        torch.cuda.synchronize()
        for l in range(s.NL):
            assert np.array_equal(out[l][0].cpu().numpy(), byte[l][sel]), (r, l)

    away = np.concatenate([np.arange(p * s.P, p * s.P + s.P) for p in range(s.full)
                           if s.page_map[0, p] < 0])
    away = away[away < L - s.T]
    first, second = s.rng.choice(away, k, replace=False), s.rng.choice(away, k, replace=False)
    second[:20] = first[:20]  # hits among its rows
    fill(0, resolve(0, first))
    slots(0)
    pending = resolve(0, second)
    assert pending["count"].item() > 0
    # a page of the pending rows becomes ready
    p = int(second[-1]) // s.P
    status = torch.full((1,), 77, **i32)
    s.ctx.restore_pages(1, ints(0), ints(p), ints(int(np.nonzero(s.refs == 0)[0][0])), status)
    s.ctx.fork_requests(1, ints(0), ints(1))
    s.ctx.fork_requests(1, ints(1), ints(2))
    torch.cuda.synchronize()
    assert status.item() == 0
    for r in (1, 2):
        slots(r)
    fill(0, pending)  # the source's own
    for r in (0, 1, 2):
        slots(r)
        got = resolve(r, second)
        assert got["count"].item() == 0
        rows(r, second, got)
    # the copy of a request that is resolved again after the fork
    third = s.rng.choice(away, k, replace=False)
    got = resolve(2, third)
    s.ctx.fork_requests(1, ints(2), ints(3))
    slots(3)
    fill(2, got)
    rows(2, third, got)
    got = resolve(3, third)
    assert got["count"].item() == 0
    rows(3, third, got)


@pytest.mark.parametrize("seed,P,R,NL", [(41, 64, 1152, 2), (42, 129, 256, 1), (43, 128, 256, 3),
                                          (44, 200, 1152, 1), (45, 16, 4096, 2)])
def test_long_pages(seed, P, R, NL):
    """Copies and compaction of pages that several workgroups share: pages of
    one piece and a little more, of exactly one, of several."""
    s = State(seed, P=P, R=R, NL=NL, H=5 * P + 3, ready=0.7, spare=9)
    s.ctx.fork_requests(1, ints(0), ints(3))
    s.fork(0, 3)
    free = np.nonzero(s.refs == 0)[0]
    held = [(r, p) for r in range(s.n_req) for p in range(s.full) if s.page_map[r, p] >= 0]
    take = [(r, p, int(ph)) for (r, p), ph in zip(held, free[-4:])]
    assert len(take) == 4
    status = torch.full((4,), 77, dtype=torch.int32, device="cuda")
    s.ctx.copy_pages(4, *[ints(*col) for col in zip(*take)], status)
    for r, p, ph in take:
        old = s.page_map[r, p]
        for l in range(NL):
            s.pool[l][ph] = s.pool[l][old]
        s.refs[old] -= 1
        s.refs[ph] += 1
        s.page_map[r, p] = ph
    s.check()
    assert status.cpu().tolist() == [0] * 4
    s.ctx.release_requests(2, ints(0, 1))
    s.release(0)
    s.release(1)
    moves = torch.zeros(s.pages, 2, dtype=torch.int32, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    for most in (2, s.pages):
        s.ctx.compact_pool(most, moves, n, s.ws)
        plan = s.compact(most)
        s.check()
        assert n.item() == len(plan) and moves.cpu().tolist()[:len(plan)] == [list(m) for m in plan]


def test_captured_and_replayed():
    """Release, fork and compaction as one graph, replayed over changing state."""
    s = State(31, n_req=8, users=4, ready=0.6)
    src, dst = ints(0, 1), ints(5, 6)
    moves = torch.zeros(s.pages, 2, dtype=torch.int32, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        s.ctx.release_requests(2, dst)
        s.ctx.compact_pool(s.pages, moves, n, s.ws)
        s.ctx.fork_requests(2, src, dst)
    for step in range(4):
        src.copy_(ints(step % 4, (step + 2) % 4))
        g.replay()
        s.release(5)
        s.release(6)
        s.compact(s.pages)
        s.fork(step % 4, 5)
        s.fork((step + 2) % 4, 6)
        s.check()
        if step == 1:
            s.ctx.release_requests(1, ints(3))
            s.release(3)


def test_refusals():
    from hierarchical_sparse_kv_resolve_amd import KvrError
    s = State(41)
    one = ints(0)
    status = ints(0)
    with pytest.raises(KvrError, match="status is required"):
        s.ctx.copy_pages(1, one, one, one, None)
    with pytest.raises(KvrError, match="page lists"):
        s.ctx.copy_pages(1, one, None, one, status)
    with pytest.raises(KvrError, match="req_ids"):
        s.ctx.release_requests(1, None)
    with pytest.raises(ValueError, match="dst_ids: 4 bytes"):
        s.ctx.fork_requests(2, ints(0, 1), one)
    with pytest.raises(TypeError, match="expected a GPU tensor"):
        s.ctx.fork_requests(1, one.cpu(), one)
    with pytest.raises(TypeError, match="src_ids: expected int32"):
        s.ctx.fork_requests(1, one.long(), one)
    with pytest.raises(TypeError, match="phys: expected int32"):
        s.ctx.copy_pages(1, one, one, one.float(), status)
    with pytest.raises(ValueError, match="refs: "):
        s.ctx.bind_page_refs(s.dev["refs"][:-1])
    moves = torch.zeros(s.pages, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(KvrError, match="workspace has"):
        s.ctx.compact_pool(s.pages, moves, one, s.ws[:-4])
    with pytest.raises(KvrError, match="workspace has 0"):
        s.ctx.list_free_pages(moves, one, None)
    with pytest.raises(KvrError, match="negative max_moves"):
        s.ctx.compact_pool(-1, moves, one, s.ws)
    with pytest.raises(ValueError, match="moves: "):
        s.ctx.compact_pool(s.pages, moves[:-1].contiguous(), one, s.ws)
    s.ctx.bind_page_refs(None)
    for call in (lambda: s.ctx.fork_requests(1, one, ints(1)), lambda: s.ctx.count_page_refs(),
                 lambda: s.ctx.release_requests(1, one),
                 lambda: s.ctx.copy_pages(1, one, one, one, status),
                 lambda: s.ctx.compact_pool(1, moves, one, s.ws)):
        with pytest.raises(KvrError, match="not bound"):
            call()
    s.check()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_pack_resolve_fork_compact_attend(fmt):
    """A request's rows are packed into its places, resolved and attended to; a
    fork of it, and both after a compaction, attend to the same rows with the
    same result, from locations and from gathered rows; a decoded row packed,
    appended and selected changes only its own request."""
    from hierarchical_sparse_kv_resolve_amd import Context
    rng = np.random.default_rng(51)
    n_req, H, P, T, B, k, heads = 3, 520, 16, 30, 150, 140, 16
    R, npg, full = ref.row_bytes(fmt, 512, 64), -(-520 // 16), 520 // 16
    pages = 40
    ctx = Context(n_req=n_req, n_layers=1, history_rows=H, max_new_rows=4, page_rows=P, tail_rows=T,
                  hot_slots=B, row_bytes=R, sel_cap=k, pool_pages=pages)
    i32 = dict(dtype=torch.int32, device="cuda")
    # pack the history of request 0 and put its rows where they belong
    latent = torch.from_numpy(rng.standard_normal((H, 512))).bfloat16().cuda()
    rope = torch.from_numpy(rng.standard_normal((H, 64))).bfloat16().cuda()
    rows = torch.zeros(H, R, dtype=torch.uint8, device="cuda")
    w = torch.ones(512, device="cuda")
    ctx.pack_rows(H, latent, rope, rows, fmt=fmt, d_v=512, d_rope=64, weight=w, eps=1e-6)
    keys = ref.unpack(rows, fmt, 512, 64)
    pm = torch.full((n_req, npg), -1, dtype=torch.int32)
    ready = rng.permutation(full)[:16]
    phys = rng.permutation(np.arange(20, pages))[:16]  # the low pages are free
    pm[0, ready] = torch.from_numpy(phys.astype(np.int32))
    hv = (pm < 0).to(torch.uint8)
    hv[1:] = 0
    pool = torch.full((pages, P, R), POISON, dtype=torch.uint8, device="cuda")
    for p, ph in zip(ready, phys):
        pool[ph] = rows[p * P:(p + 1) * P]
    host = torch.full((n_req, H + 4, R), POISON, dtype=torch.uint8).pin_memory()
    for p in range(npg):
        if hv[0, p]:
            host[0, p * P:min(H, p * P + P)] = rows[p * P:min(H, p * P + P)].cpu()
    tail = torch.full((n_req, T, R), POISON, dtype=torch.uint8, device="cuda")
    for pos in range(H - T, H):
        tail[0, pos % T] = rows[pos]
    hot = torch.full((n_req, B, R), POISON, dtype=torch.uint8, device="cuda")
    L = torch.zeros(n_req, **i32)
    meta = [L, pm.cuda(), hv.cuda(), torch.full((n_req, B), -1, **i32),
            torch.zeros(n_req, B, **i32), torch.zeros(n_req, **i32)]
    refs = torch.zeros(pages, **i32)
    ctx.bind_metadata(*meta)
    ctx.bind_layer(0, tail, pool, hot, host)
    ctx.init_state()
    ctx.bind_page_refs(refs)
    ctx.count_page_refs()
    ctx.release_requests(2, ints(1, 2))
    q1 = torch.from_numpy(rng.standard_normal((1, 1, heads, 576))).bfloat16().cuda()
    ws = torch.empty(ctx.attend_workspace(n_req, 1, heads, 512, k), dtype=torch.uint8, device="cuda")
    pws = torch.empty(ctx.pool_workspace(), dtype=torch.uint8, device="cuda")

    def step(reqs, sel):
        """Resolve, attend from locations and from the gathered buffer."""
        n = len(reqs)
        ids = ints(*reqs)
        sel_d = torch.from_numpy(np.tile(sel.astype(np.int32), (n, 1))).cuda()
        loc = torch.full((n, k), -1, **i32)
        fills, fc, st = torch.zeros(n, B, 2, **i32), torch.zeros(n, **i32), torch.zeros(n, **i32)
        ctx.resolve_rows(n, ids, sel_d, None, k, loc, fills, fc, 0, st)
        q = q1.expand(n, 1, heads, 576)
        out = torch.zeros(n, 1, heads, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(n, 1, heads, device="cuda")
        ctx.attend_rows(0, n, ids, q, out, fmt=fmt, d_v=512, d_rope=64, scale=0.07, stride=k,
                        loc=loc, lse=lse, workspace=ws)
        buf = torch.zeros(n, k, R, dtype=torch.uint8, device="cuda")
        ctx.gather_rows([0], n, ids, loc, None, k, [buf])
        out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
        ctx.attend_rows(0, n, ids, q, out2, fmt=fmt, d_v=512, d_rope=64, scale=0.07, stride=k,
                        rows=buf, lse=lse2, workspace=ws)
        torch.cuda.synchronize()
        assert (st == 0).all() and torch.equal(out, out2) and torch.equal(lse, lse2)
        want = ref.attend(q1[0, 0].cpu(), keys[sel], 512, 0.07)
        for i in range(n):
            # 2^-8 for the probabilities, 2^-8 for the result, 2^-9 for 32-bit sums
            o = out[i, 0].cpu().double()
            assert ((o - want[0]).abs() <= 2.0 ** -8 * (1.5 * want[2] + want[0].abs())).all()
            assert ((lse[i, 0].cpu().double() - want[1]).abs() < 1e-3).all()
        return out, lse

    # every place, with a repeat
    first = np.r_[rng.choice(H, k - 1, replace=False), 519]
    a, _ = step([0], first)
    ctx.fork_requests(2, ints(0, 0), ints(1, 2))
    b, _ = step([0, 1, 2], first)
    assert torch.equal(b[0], b[1]) and torch.equal(b[0], b[2])
    second = rng.choice(H, k, replace=False)
    c, _ = step([2, 1], second)
    moves, n_moves = torch.zeros(pages, 2, **i32), torch.zeros(1, **i32)
    ctx.compact_pool(pages, moves, n_moves, pws)
    torch.cuda.synchronize()
    assert n_moves.item() == 16 and int(meta[1].max()) == 15
    assert refs.cpu().tolist() == [3] * 16 + [0] * (pages - 16)
    pool[16:] = POISON  # nothing reads the freed pages
    d, _ = step([1, 0, 2], second)
    assert torch.equal(d[0], c[1]) and torch.equal(d[2], c[0])
    # a decoded row of request 1
    new = torch.zeros(1, 1, R, dtype=torch.uint8, device="cuda")
    lat2 = torch.from_numpy(rng.standard_normal((1, 576))).bfloat16().cuda()
    ctx.pack_rows(1, lat2[:, :512], lat2[:, 512:], new, fmt=fmt, d_v=512, d_rope=64, weight=w,
                  eps=1e-6)
    ctx.append_rows(1, ints(1), new)
    keys = torch.cat([keys, ref.unpack(new[0], fmt, 512, 64)])
    third = np.r_[second[:k - 1], H]
    step([1], third)
    ctx.release_requests(1, ints(0))
    step([1], third)
    keys = keys[:H]
    step([2], first)
