"""Paged key-value cache, restated plainly for the tests: the attention of one
token in float64, and the page calls as loops over Python lists.  Shares no
code with the CUDA path."""

from __future__ import annotations

import numpy as np

__all__ = ["decode", "PageModel"]


def decode(q, k_pages, v_pages, table, lengths, scale):
    """q [S, H, d], pools [pages, H_kv, R, d], all float64 -> (O [S, H, d], L [S, H], A [S, H], V [S, H]).

    A is the largest scale * sum_c |q_c k_jc| over the visible rows and V the
    largest |v_jc|: what rounding errors of the scores and of the weighted sum
    are measured in.  Rows on pages that do not exist are not visible."""
    S, H, d = q.shape
    pages, hk, rows, _ = k_pages.shape
    o, L = np.zeros((S, H, d)), np.full((S, H), np.inf)
    A, V = np.zeros((S, H)), np.zeros((S, H))
    for s in range(S):
        at = []
        for j in range(min(max(int(lengths[s]), 0), rows * table.shape[1])):
            p = int(table[s, j // rows])
            if 0 <= p < pages:
                at.append((p, j % rows))
        if not at:
            continue
        pp, rr = np.array([a[0] for a in at]), np.array([a[1] for a in at])
        for h in range(H):
            g = h // (H // hk)
            k, v = k_pages[pp, g, rr], v_pages[pp, g, rr]
            x = scale * (k @ q[s, h])
            m = x.max()
            e = np.exp(x - m)
            o[s, h] = (e @ v) / e.sum()
            L[s, h] = m + np.log(e.sum())
            A[s, h] = scale * (np.abs(k) @ np.abs(q[s, h])).max()
            V[s, h] = np.abs(v).max()
    return o, L, A, V


class PageModel:
    """table (list of lists, -1 behind a sequence's pages), lengths, refs."""

    def __init__(self, pages, rows, sequences, columns):
        self.rows, self.columns = rows, columns
        self.table = [[-1] * columns for _ in range(sequences)]
        self.lengths = [0] * sequences
        self.refs = [0] * pages

    def held(self, n):
        return -(-n // self.rows)

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def extend(self, n_new):
        free, plan = self.free_pages(), []
        for s, more in enumerate(n_new):
            n = self.lengths[s]
            if more < 0 or self.held(n + more) > self.columns or n + more > self.rows * self.columns:
                return None
            plan.append((s, list(range(self.held(n), self.held(n + more)))))
        if sum(len(c) for _, c in plan) > len(free):
            return None
        start = list(self.lengths)
        for s, columns in plan:
            for c in columns:
                p = free.pop(0)
                self.table[s][c] = p
                self.refs[p] = 1
            self.lengths[s] += n_new[s]
        return start

    def fork(self, src, dst):
        S = len(self.lengths)
        if any(not 0 <= i < S for i in list(src) + list(dst)):
            return None
        if len(set(dst)) < len(dst) or set(src) & set(dst) or any(self.lengths[b] for b in dst):
            return None
        free = self.free_pages()
        if sum(self.lengths[a] % self.rows > 0 for a in src) > len(free):
            return None
        moves = []
        for a, b in zip(src, dst):
            n = self.lengths[a]
            for c in range(n // self.rows):
                self.table[b][c] = self.table[a][c]
                self.refs[self.table[a][c]] += 1
            if n % self.rows:
                c, p = n // self.rows, free.pop(0)
                moves.append((self.table[a][c], p, n % self.rows))
                self.table[b][c] = p
                self.refs[p] = 1
            else:
                moves.append((-1, -1, -1))
            self.lengths[b] = n
        return moves

    def free(self, sequences):
        for s in sequences:
            if s < 0:
                continue
            for c in range(self.held(self.lengths[s])):
                self.refs[self.table[s][c]] -= 1
                self.table[s][c] = -1
            self.lengths[s] = 0

    def compact(self):
        used = [p for p, r in enumerate(self.refs) if r > 0]
        n = len(used)
        holes = [p for p in range(n) if self.refs[p] == 0]
        movers = [p for p in used if p >= n]
        to = {p: p for p in used}
        to.update(zip(movers, holes))
        refs = [0] * len(self.refs)
        for p in used:
            refs[to[p]] = self.refs[p]
        self.refs = refs
        self.table = [[to[p] if p >= 0 else -1 for p in row] for row in self.table]
        return [(a, b, self.rows) for a, b in zip(movers, holes)]
