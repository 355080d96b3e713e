"""Bounds of pages, the choice by them and the pages' bookkeeping from their definitions, on the host."""
from __future__ import annotations

import math

import numpy as np
import torch


def power(top):
    """The least power of two s >= 2^-100 with top <= 127 s."""
    s = 2.0 ** -100
    if top > 127 * s:
        s = 2.0 ** (math.frexp(top)[1] - 8)
        while top > 127 * s:
            s *= 2
    return s


def finite(x):
    """NaN counts as not there (None), infinities as the largest finite number."""
    return None if math.isnan(x) else max(-3.4028234663852886e38, min(3.4028234663852886e38, x))


def page_bounds(keys):
    """keys [slots, dim] (numpy float64): (lo, hi, scale)."""
    with np.errstate(invalid="ignore"):
        clean = np.clip(keys, -3.4028234663852886e38, 3.4028234663852886e38)
    lo = np.array([0.0 if np.isnan(c).all() else np.nanmin(c) for c in clean.T])
    hi = np.array([0.0 if np.isnan(c).all() else np.nanmax(c) for c in clean.T])
    s = power(max(np.abs(lo).max(), np.abs(hi).max()))
    return np.floor(lo / s), np.ceil(hi / s), s


def page_score(queries, lo, hi, s):
    """queries [group, dim]; the largest over the group, in whole numbers times powers of two."""
    best = -math.inf
    for q in queries:
        q = np.array([0.0 if math.isnan(x) else finite(x) for x in q])
        t = power(np.abs(q).max())
        z = np.rint(q / t)
        best = max(best, float(np.maximum(z * lo, z * hi).sum()) * s * t)
    return best


def choose(scores, keep, first, recent):
    """Indexes of the pages kept, in order."""
    n = len(scores)
    if n <= keep:
        return list(range(n))
    middle = sorted(range(first, n - recent), key=lambda i: (-scores[i], i))[:keep - first - recent]
    return sorted(list(range(first)) + middle + list(range(n - recent, n)))


class Pool:
    """uses, lists and lengths as the calls leave them."""

    def __init__(self, uses, page, width):
        self.uses, self.page, self.width, self.error = list(uses), page, width, False

    def pages_of(self, n):
        return -(-n // self.page)

    def take(self, wants):
        """wants[b] pages for each in turn: lists of pages, None where they are not there."""
        free = [p for p, u in enumerate(self.uses) if u == 0]
        at, out = 0, []
        for w in wants:
            got = free[at:at + w] if at + w <= len(free) else None
            at += w
            if got is None:
                self.error = True
            else:
                for p in got:
                    self.uses[p] = 1
            out.append(got)
        return out

    def grow(self, table, lengths, tokens):
        wants = []
        for b, (n, t) in enumerate(zip(lengths, tokens)):
            if not 0 <= n <= self.width * self.page or t < 0 or n + t > self.width * self.page:
                self.error = True
                wants.append(-1)
            else:
                wants.append(self.pages_of(n + t) - self.pages_of(n))
        got = self.take([max(w, 0) for w in wants])
        for b, (w, g) in enumerate(zip(wants, got)):
            if w < 0 or g is None:
                continue
            first = self.pages_of(lengths[b])
            table[b][first:first + w] = g
            lengths[b] += tokens[b]

    def fork(self, table, lengths, parents, to_table, to_lengths):
        """Returns the copies: (page from, page to, rows)."""
        take = []
        for p in parents:
            n = 0
            if p != -1:
                if not 0 <= p < len(lengths) or self.pages_of(lengths[p]) > len(to_table[0]):
                    self.error = True
                else:
                    n = lengths[p]
            take.append(n)
        got = self.take([1 if n % self.page else 0 for n in take])
        copies = []
        for c, (n, g) in enumerate(zip(take, got)):
            full = n // self.page
            for i in range(full):
                to_table[c][i] = table[parents[c]][i]
                self.uses[to_table[c][i]] += 1
            to_lengths[c] = n if g is not None else full * self.page
            if g:
                to_table[c][full] = g[0]
                copies.append((table[parents[c]][full], g[0], n % self.page))
        return copies

    def free(self, table, lengths):
        for b, n in enumerate(lengths):
            for i in range(self.pages_of(n)):
                self.uses[table[b][i]] -= 1
            lengths[b] = 0

    def compact(self, table, lengths):
        """Returns the moves {from: to} and the number of pages in use."""
        n = sum(u > 0 for u in self.uses)
        above = [p for p in range(n, len(self.uses)) if self.uses[p] > 0]
        moves = dict(zip(above, [p for p in range(n) if self.uses[p] == 0]))
        for a, z in moves.items():
            self.uses[z], self.uses[a] = self.uses[a], 0
        for b, m in enumerate(lengths):
            for i in range(self.pages_of(m)):
                table[b][i] = moves.get(table[b][i], table[b][i])
        return moves, n


def as_list(t):
    return t.cpu().tolist()


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")
