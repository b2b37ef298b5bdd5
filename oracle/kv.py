"""Paged 8-bit key/value cache and the attention that reads it (oracle side, fp64, numpy).

The pages name no cache; the formats are those of the other outputs (E4M3
codes, E8M0 scale bytes).  Readings, as include/rn.h states them:

* row starts[b] + i of a call with n rows of sequence b is position
  lens[b] - n + i; block i of 64 positions stands in page table[b, i]; a page
  number that is none, a block past the table and a negative position mean
  that the position is not cached;
* write: e = the smallest exponent with amax <= 448 2^e, clamped to [-120, 119],
  code = E4M3(x 2^-e); a begun page keeps the larger exponent, and its old
  codes become E4M3(value 2^(e' - e));
* attention: s = scale q.k, c tanh(s / c), + slope (j - p); softmax over the
  positions seen; no position: 0 and -inf.

Everything here goes position by position, without the library's tiling.
"""
from __future__ import annotations

import numpy as np

from .formats import e4m3_decode, e4m3_encode

PAGE = 64
E_MIN, E_MAX = -120, 119


def exponent(values) -> int:
    a = np.abs(np.asarray(values, dtype=np.float64)).ravel()
    a = a[np.isfinite(a)]
    top = a.max() if a.size else 0.0
    e = E_MIN
    while e < E_MAX and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def byte_exponent(byte) -> int:
    return int(min(max(int(byte) - 127, E_MIN), E_MAX))


class Cache:
    """k [pages, heads, 64, dim], v [pages, heads, dim, 64], ks / vs [pages, heads], all uint8."""

    def __init__(self, k, v, ks, vs):
        self.k, self.v, self.ks, self.vs = (np.array(a, dtype=np.uint8) for a in (k, v, ks, vs))
        self.pages, self.heads, _, self.dim = self.k.shape

    def page(self, table, b, position) -> int:
        """The page of a position, -1 if it is not cached."""
        if position < 0 or position // PAGE >= table.shape[1]:
            return -1
        p = int(table[b, position // PAGE])
        return p if 0 <= p < self.pages else -1

    def columns(self, which, page, h):
        """The codes of a page and head as [64, dim], a view."""
        return self.k[page, h] if which == "k" else self.v[page, h].T

    def scales(self, which):
        return self.ks if which == "k" else self.vs


def rows_of(starts, lens, b):
    """(row, position) of each row of sequence b."""
    n = int(starts[b + 1]) - int(starts[b])
    return [(int(starts[b]) + i, int(lens[b]) - n + i) for i in range(n)]


def write(c: Cache, table, starts, lens, k, v) -> Cache:
    """The cache after the rows k, v [tokens, heads, dim] have been written."""
    c = Cache(c.k, c.v, c.ks, c.vs)
    for b in range(len(lens)):
        blocks = {}
        for row, pos in rows_of(starts, lens, b):
            if c.page(table, b, pos) >= 0:
                blocks.setdefault(pos // PAGE, []).append((row, pos % PAGE))
        for blk, rows in blocks.items():
            page, first = int(table[b, blk]), rows[0][1]
            for which, x in (("k", k), ("v", v)):
                for h in range(c.heads):
                    new = np.stack([np.asarray(x[r, h], dtype=np.float64) for r, _ in rows])
                    e, cols = exponent(new), c.columns(which, page, h)
                    if first > 0:
                        old = byte_exponent(c.scales(which)[page, h])
                        if e > old:
                            cols[:first] = e4m3_encode(e4m3_decode(cols[:first]) * 2.0 ** (old - e))
                        e = max(e, old)
                    for (_, at), y in zip(rows, new):
                        cols[at] = e4m3_encode(y * 2.0 ** -e)
                    c.scales(which)[page, h] = e + 127
    return c


def values(c: Cache, which, page, h) -> np.ndarray:
    return e4m3_decode(c.columns(which, page, h)) * 2.0 ** byte_exponent(c.scales(which)[page, h])


def sequence(c: Cache, table, b, n, which) -> tuple:
    """Positions 0 .. n - 1 of a sequence: values [n, heads, dim] (0 where not cached), cached [n]."""
    out, there = np.zeros((n, c.heads, c.dim)), np.zeros(n, dtype=bool)
    for blk in range((n + PAGE - 1) // PAGE):
        page = c.page(table, b, blk * PAGE)
        m = min(PAGE, n - blk * PAGE)
        if page >= 0:
            there[blk * PAGE:blk * PAGE + m] = True
            for h in range(c.heads):
                out[blk * PAGE:blk * PAGE + m, h] = values(c, which, page, h)[:m]
    return out, there


def read(c: Cache, table, starts, lens, tokens) -> tuple:
    """(k, v) [tokens, heads, dim], NaN in rows of no sequence."""
    out = []
    for which in "kv":
        x = np.full((tokens, c.heads, c.dim), np.nan)
        for b in range(len(lens)):
            full, _ = sequence(c, table, b, max(int(lens[b]), 0), which)
            for row, pos in rows_of(starts, lens, b):
                x[row] = full[pos] if pos >= 0 else 0.0
        out.append(x)
    return tuple(out)


def attention(q, c: Cache, table, starts, lens, scale, causal=True, window=0, softcap=0.0, slopes=None) -> dict:
    """out [tokens, q heads, dim] and lse, NaN in rows of no sequence; and what bounds of their errors
    need: "pv" = sum p |v|, "big" = max over the seen of (|q| . |k|) scale, "spread" = max p 2^e sum
    |code| (e and code of the values), "seen" = positions seen."""
    q = np.asarray(q, dtype=np.float64)
    T, heads, D = q.shape
    group = heads // c.heads
    r = {"out": np.full(q.shape, np.nan), "lse": np.full((T, heads), np.nan), "pv": np.zeros(q.shape),
         "big": np.zeros((T, heads)), "spread": np.zeros(q.shape), "seen": np.zeros((T, heads), dtype=np.int64)}
    for b in range(len(lens)):
        n = max(int(lens[b]), 0)
        k, there = sequence(c, table, b, n, "k")
        v, _ = sequence(c, table, b, n, "v")
        unit = np.ones((n, c.heads))
        for j in range(n):
            if there[j]:
                unit[j] = [2.0 ** byte_exponent(x) for x in c.vs[c.page(table, b, j)]]
        pos = np.arange(n)
        for row, p in rows_of(starts, lens, b):
            sees = there & (pos <= p if causal else True) & (pos > p - window if window > 0 else True)
            for h in range(heads):
                g = h // group
                r["out"][row, h], r["lse"][row, h] = 0.0, -np.inf
                if not sees.any():
                    continue
                s = scale * (k[sees, g] @ q[row, h])
                r["big"][row, h] = scale * (np.abs(k[sees, g]) @ np.abs(q[row, h])).max()
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s + float(slopes[h]) * (pos[sees] - p)
                    r["big"][row, h] = max(r["big"][row, h], abs(float(slopes[h])) * (np.abs(pos[sees] - p).max()))
                top = s.max()
                w = np.exp(s - top)
                r["lse"][row, h] = top + np.log(w.sum())
                w = w / w.sum()
                r["out"][row, h] = w @ v[sees, g]
                r["pv"][row, h] = w @ np.abs(v[sees, g])
                u = unit[sees, g]
                r["spread"][row, h] = (w * u).max() * np.abs(v[sees, g] / u[:, None]).sum(0)
                r["seen"][row, h] = sees.sum()
    return r
