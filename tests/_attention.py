"""Plain 64-bit attention, page bookkeeping on lists, and error bounds.

Roundings are counted as half a step relative to the value: EPS32 = 2^-24 for
float32, EPS16 = 2^-8 for bfloat16.  The bounds are sums over a result's
terms, each with the relative error it can have."""
from __future__ import annotations

import math

import numpy as np
import torch

EPS32 = 2.0 ** -24
EPS16 = 2.0 ** -8


def visible(nq: int, nk: int, window: int, sinks: int) -> torch.Tensor:
    pos = torch.arange(nk - nq, nk)[:, None]
    j = torch.arange(nk)[None]
    see = j <= pos
    if window:
        see &= (pos - j < window) | (j < sinks)
    return see


def attention(q, k, v, see, scale: float):
    """q [n, D], k, v [m, D] float64, see [n, m] -> (o, lse, P); empty rows 0, -inf."""
    s = (q @ k.T) * scale
    s = torch.where(see, s, -math.inf)
    lse = torch.logsumexp(s, 1)
    P = torch.where(see, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None]), 0.0)
    return P @ v, lse, P


def score_error(q, k, scale: float, depth: float):
    """Bound of |error| of scale * q . k summed in float32, per pair: every
    product and partial sum rounded (depth of them on a term's way, 2^-23 each
    as the tensor cores may truncate), the scaling and the split terms' rest."""
    return (depth + 4) * 2.0 ** -23 * scale * (q.abs() @ k.abs().T)


class PageModel:
    """Tables, lengths and reference counts on lists, one sequence after the other."""

    def __init__(self, num_pages, page_size, max_seqs, max_pages):
        self.ps, self.n = page_size, num_pages
        self.tables = [[-1] * max_pages for _ in range(max_seqs)]
        self.lengths = [0] * max_seqs
        self.refs = [0] * num_pages
        self.moves = []

    def pages_of(self, n):
        return -(-n // self.ps)

    def free_pages(self):
        return [p for p in range(self.n) if self.refs[p] == 0]

    def extend(self, ids, counts):
        bad, need, seen = 0, 0, set()
        for s, c in zip(ids, counts):
            if s < 0:
                continue
            if s >= len(self.lengths) or c < 0 or s in seen:
                bad = max(bad, 3)
                continue
            seen.add(s)
            if self.lengths[s] + c > len(self.tables[s]) * self.ps:
                bad = max(bad, 2)
            else:
                need += self.pages_of(self.lengths[s] + c) - self.pages_of(self.lengths[s])
        if bad:
            return bad
        free = self.free_pages()
        if need > len(free):
            return 1
        for s, c in zip(ids, counts):
            if s < 0:
                continue
            for j in range(self.pages_of(self.lengths[s]), self.pages_of(self.lengths[s] + c)):
                self.tables[s][j] = free.pop(0)
                self.refs[self.tables[s][j]] = 1
            self.lengths[s] += c
        return 0

    def free(self, ids):
        for s in ids:
            if s < 0 or s >= len(self.lengths):
                continue
            for j in range(self.pages_of(self.lengths[s])):
                self.refs[self.tables[s][j]] -= 1
                self.tables[s][j] = -1
            self.lengths[s] = 0

    def fork(self, src, dst):
        self.moves = []
        pairs = [(a, b) for a, b in zip(src, dst) if a >= 0 and b >= 0]
        m = len(self.lengths)
        if any(a >= m or b >= m for a, b in pairs):
            return 3
        if len({b for _, b in pairs}) != len(pairs) or {a for a, _ in pairs} & {b for _, b in pairs}:
            return 3
        if any(self.lengths[b] for _, b in pairs):
            return 3
        free = self.free_pages()
        if sum(self.lengths[a] % self.ps != 0 for a, _ in pairs) > len(free):
            return 1
        for a, b in pairs:
            full = self.lengths[a] // self.ps
            for j in range(full):
                self.tables[b][j] = self.tables[a][j]
                self.refs[self.tables[a][j]] += 1
            if self.lengths[a] % self.ps:
                self.tables[b][full] = free.pop(0)
                self.refs[self.tables[b][full]] = 1
                self.moves.append((self.tables[a][full], self.tables[b][full]))
            self.lengths[b] = self.lengths[a]
        return 0

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in range(live, self.n) if self.refs[p] > 0]
        self.moves = list(zip(movers, holes))
        to = dict(self.moves)
        for a, b in self.moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.tables = [[to.get(p, p) for p in row] for row in self.tables]
        return live

    def check(self, tables, lengths, refs):
        assert np.array_equal(tables.cpu().numpy(), np.array(self.tables, np.int32))
        assert lengths.cpu().tolist() == self.lengths
        assert refs.cpu().tolist() == self.refs
