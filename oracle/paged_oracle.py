"""CPU oracle of the paged K/V cache: attention in FP64 over rows gathered through a page table, and
the operations on pages as plain list walks.

Written from the definitions in include/tl_paged.h; test infrastructure only.
"""
from __future__ import annotations

import numpy as np


def rows_of(pool, table_row, head: int, n: int) -> np.ndarray:
    """Positions 0 .. n-1 of one sequence and K/V head: pool [n_pages, kv, page, hd] -> float64 [n, hd]."""
    page = pool.shape[2]
    out = np.zeros((n, pool.shape[3]))
    for pos in range(0, n, page):
        m = min(page, n - pos)
        out[pos:pos + m] = pool[table_row[pos // page], head, :m]
    return out


def attend(q, k, v, scale: float, last=None):
    """Queries q [n, hd] over rows k, v [m, hd]; query i attends rows 0 .. last[i] (None: all).  Returns
    (out [n, hd], sum_c p_c |v_c| [n, hd], max_c sum_d |q_d k_cd| [n]): the result and what bounds its
    rounding errors.  A query that attends nothing gives zeros."""
    q = np.asarray(q, np.float64)
    out, mag, reach = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[0])
    for i in range(q.shape[0]):
        m = k.shape[0] if last is None else min(max(int(last[i]) + 1, 0), k.shape[0])
        if m <= 0:
            continue
        s = scale * (k[:m] @ q[i])
        p = np.exp(s - s.max())
        p /= p.sum()
        out[i], mag[i] = p @ v[:m], p @ np.abs(v[:m])
        reach[i] = (np.abs(k[:m]) @ np.abs(q[i])).max()
    return out, mag, reach


def decode(pool_k, pool_v, table, q, kv_len, seqs, scale):
    """q [lanes, heads, hd]; the three arrays of attend, [lanes, heads, ...]."""
    lanes, heads, hd = q.shape
    kv = pool_k.shape[1]
    res = [np.zeros((lanes, heads, hd)), np.zeros((lanes, heads, hd)), np.zeros((lanes, heads))]
    for b in range(lanes):
        for h in range(heads):
            g = h // (heads // kv)
            k = rows_of(pool_k, table[seqs[b]], g, kv_len[b])
            v = rows_of(pool_v, table[seqs[b]], g, kv_len[b])
            for r, x in zip(res, attend(q[b, h][None], k, v, scale)):
                r[b, h] = x[0]
    return res


def prompt(pool_k, pool_v, table, q, cu_q, kv_len, seqs, scale):
    """q [rows, heads, hd] packed; the three arrays of attend, [rows, heads, ...]; rows outside every lane are NaN."""
    rows, heads, hd = q.shape
    kv = pool_k.shape[1]
    res = [np.full((rows, heads, hd), np.nan), np.full((rows, heads, hd), np.nan), np.full((rows, heads), np.nan)]
    for b in range(len(kv_len)):
        lo, hi = cu_q[b], cu_q[b + 1]
        last = kv_len[b] - (hi - lo) + np.arange(hi - lo)
        for h in range(heads):
            g = h // (heads // kv)
            k = rows_of(pool_k, table[seqs[b]], g, kv_len[b])
            v = rows_of(pool_v, table[seqs[b]], g, kv_len[b])
            for r, x in zip(res, attend(q[lo:hi, h], k, v, scale, last)):
                r[lo:hi, h] = x
    return res


class Pages:
    """The page table and counts of a cache, and what the operations do to them.  Each operation returns the page
    copies it makes, [(source, destination)], and notes in ``flags`` what the library records as its status."""

    def __init__(self, n_pages, page, max_seqs, max_pages):
        self.page, self.n_pages, self.max_seqs, self.max_pages = page, n_pages, max_seqs, max_pages
        self.table = np.full((max_seqs, max_pages), -1, np.int32)
        self.refs = np.zeros(n_pages, np.int32)
        self.flags = set()

    def _count(self, n):
        return -(-n // self.page)

    def copy(self, src, dst):
        moves = []
        for i, (a, b) in enumerate(zip(src, dst)):
            ok = 0 <= a < self.n_pages and 0 <= b < self.n_pages and b not in dst[:i] and a not in dst
            moves += [(a, b)] if ok else []
            self.flags |= set() if ok else {"range"}
        return moves

    def fork(self, src, dst, n_tokens):
        for i, (a, d, n) in enumerate(zip(src, dst, n_tokens)):
            ok = 0 <= a < self.max_seqs and 0 <= d < self.max_seqs and 0 <= n <= self.max_pages * self.page
            ok = ok and a not in dst and d not in dst[:i] and (self.table[d] < 0).all()
            ok = ok and (self.table[a, :self._count(n)] >= 0).all()
            if not ok:
                self.flags.add("range")
                continue
            for j in range(self._count(n)):
                self.table[d, j] = self.table[a, j]
                self.refs[self.table[a, j]] += 1
        return []

    def reserve(self, seqs, ctx, new):
        before, plan, want = self.refs.copy(), [], 0
        free = [p for p in range(self.n_pages) if before[p] == 0]
        moves = []
        for i, (s, c, n) in enumerate(zip(seqs, ctx, new)):
            ok = 0 <= s < self.max_seqs and c >= 0 and n >= 0 and c + n <= self.max_pages * self.page and s not in seqs[:i]
            if not ok:
                self.flags.add("range")
                continue
            entries = range(c // self.page, self._count(c + n)) if n else []
            plan.append((s, c, [j for j in entries if self.table[s, j] < 0 or before[self.table[s, j]] > 1]))
        for s, c, entries in plan:
            if want + len(entries) > len(free):
                self.flags.add("full")
                break
            for j in entries:
                was, to = self.table[s, j], free[want]
                want += 1
                self.table[s, j], self.refs[to] = to, 1
                if was >= 0:
                    self.refs[was] -= 1
                    if j * self.page < c:
                        moves.append((int(was), to))
        return moves

    def free(self, seqs, keep=None):
        for i, s in enumerate(seqs):
            k = 0 if keep is None else keep[i]
            if not 0 <= s < self.max_seqs or k < 0:
                self.flags.add("range")
                continue
            for j in range(self._count(k), self.max_pages):
                if self.table[s, j] >= 0:
                    self.refs[self.table[s, j]] -= 1
                    self.table[s, j] = -1
        return []

    def compact(self):
        live = int((self.refs > 0).sum())
        moves = list(zip([p for p in range(live, self.n_pages) if self.refs[p] > 0],
                         [p for p in range(live) if self.refs[p] == 0]))
        for a, b in moves:
            self.table[self.table == a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        return moves
