"""The drafter's window in 8 bits in plain form: a ring of e4m3 codes with one
power-of-two scale for each block of 64 tokens, head, and keys or values, and
attention over it in 64 bits.  Nothing here uses the library."""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 64
NAN_CODE = 0x7F


def codes_of(x):
    """e4m3 codes (uint8) of a float64 array whose values are exact in 32 bits."""
    t = torch.from_numpy(np.ascontiguousarray(x)).float().to(torch.float8_e4m3fn)
    return t.view(torch.uint8).numpy()


def values_of(codes):
    c = torch.from_numpy(np.ascontiguousarray(codes))
    return c.view(torch.float8_e4m3fn).double().numpy()


def exponent_for(top):
    """Smallest e >= -100 with top <= 448 * 2^e."""
    e = -100
    if top > 0:
        e = max(e, math.frexp(top / 448.0)[1] - 1)
        while top > 448.0 * 2.0 ** e:
            e += 1
    return e


class Window:
    """One layer of a ring of n_req requests: keys and values [n_req][kv][C][d] as
    codes, exponents [n_req][C / 64][kv][2]."""

    def __init__(self, n_req, W, C, kv, d):
        self.n_req, self.W, self.C, self.kv, self.d = n_req, W, C, kv, d
        self.code = np.zeros((2, n_req, kv, C, d), dtype=np.uint8)
        self.exp = np.full((n_req, C // BLOCK, kv, 2), -100, dtype=np.int64)
        self.length = np.zeros(n_req, dtype=np.int64)
        self.high = np.zeros(n_req, dtype=np.int64)

    def write(self, r, k, v):
        """k, v float64 [rows, kv, d] at the positions after the rows kept."""
        a, rows = int(self.length[r]), k.shape[0]
        held = {}  # slot -> whether its row is kept
        for p in range(max(0, int(self.high[r]) - self.C), int(self.high[r])):
            held[p % self.C] = p < a
        p = a
        while p < a + rows:
            stop = min(a + rows, (p // BLOCK + 1) * BLOCK)
            b = p % self.C // BLOCK
            new = {q % self.C: q - a for q in range(p, stop)}
            for h in range(self.kv):
                both = np.zeros((2, BLOCK, self.d))
                nan_key = np.zeros(BLOCK, dtype=bool)
                for t in range(BLOCK):
                    slot = b * BLOCK + t
                    if slot in new:
                        kk, vv = k[new[slot], h], v[new[slot], h]
                        if not (np.isfinite(kk).all() and np.isfinite(vv).all()):
                            nan_key[t] = True
                            kk = np.zeros(self.d)
                            vv = np.where(np.isfinite(vv), vv, 0.0)
                        both[0, t], both[1, t] = kk, vv
                    elif held.get(slot, False):
                        for w in (0, 1):
                            x = values_of(self.code[w, r, h, slot]) * 2.0 ** self.exp[r, b, h, w]
                            if w == 0 and np.isnan(x).any():
                                nan_key[t] = True
                                x = np.zeros(self.d)
                            both[w, t] = x
                for w in (0, 1):
                    e = exponent_for(np.abs(both[w]).max())
                    self.exp[r, b, h, w] = e
                    self.code[w, r, h, b * BLOCK:(b + 1) * BLOCK] = codes_of(both[w] * 2.0 ** -e)
                self.code[0, r, h, b * BLOCK:(b + 1) * BLOCK][nan_key] = NAN_CODE
            p = stop

    def advance(self, r, rows):
        self.length[r] += rows
        self.high[r] = max(self.high[r], self.length[r])

    def rows(self, r, lo, hi):
        """Keys and values float64 [kv, hi - lo, d] of positions lo .. hi - 1."""
        slot = np.arange(lo, hi) % self.C
        e = 2.0 ** self.exp[r, slot // BLOCK].transpose(1, 0, 2)  # [kv, rows, 2]
        return (values_of(self.code[0, r][:, slot]) * e[..., :1],
                values_of(self.code[1, r][:, slot]) * e[..., 1:])

    def device_layout(self):
        """codes uint8 [n_req][C / 64][kv][2][64 * d] and scale bytes."""
        n, nb = self.n_req, self.C // BLOCK
        x = self.code.reshape(2, n, self.kv, nb, BLOCK, self.d).transpose(1, 3, 2, 0, 4, 5)
        keys = x[:, :, :, 0].reshape(n, nb, self.kv, -1)
        vals = x[:, :, :, 1].swapaxes(-1, -2).reshape(n, nb, self.kv, -1)
        return np.stack([keys, vals], 3), (self.exp + 127).astype(np.uint8)


def span(mask, length, count, j, W):
    """[lo, hi) of the positions that query j sees."""
    hi = {"causal": length + j + 1, "block": length + count, "kept": length}[mask]
    return max(0, hi - W), hi


def attend(q, k, v, scale):
    """(out, lse, spread, size) in 64 bits of the heads q [group, d] of one K/V
    head over its rows k, v [rows, d]: spread = sum p |v|, size = max of
    scale * sum |q k| (what rounding errors are measured against)."""
    if k.shape[0] == 0:
        z = np.zeros(q.shape)
        return z, np.full(q.shape[0], -np.inf), z, np.zeros(q.shape[0])
    s = q @ k.T * scale
    top = s.max(1, keepdims=True)
    e = np.exp(s - top)
    lse = (top + np.log(e.sum(1, keepdims=True)))[:, 0]
    p = np.exp(s - lse[:, None])
    return p @ v, lse, p @ np.abs(v), (np.abs(q) @ np.abs(k).T).max(1) * abs(scale)
