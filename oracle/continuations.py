"""Several continuations of one prompt, plainly and in float64: pages that sequences share, attention over a sequence's keys with
a window, a tanh cap and a distance bias, and top-k, top-p and min-p cuts with a draw. TEST INFRASTRUCTURE.

The pages have no counterpart of these; the readings are those that include/sdv.h states."""
from __future__ import annotations

import numpy as np

from .pages import CapacityError, PagePool, pages_for


class SharedPool(PagePool):
    """A page pool whose sequences can continue one another (fork) and hold pages together."""

    def holders(self, page: int) -> int:
        return sum(page in t for t in self.table)

    def fork(self, src: list, dst: list) -> list:
        """dst[i] continues src[i]; returns (source's partial page, its copy, slots filled) or None for each. All or none."""
        if len(set(dst)) != len(dst) or set(src) & set(dst) or any(self.table[d] or self.length[d] for d in dst):
            raise ValueError("a destination in use")
        partial = [self.length[s] % self.page_size for s in src]
        if sum(p > 0 for p in partial) > len(self.free):
            raise CapacityError("out of pages")
        copies = []
        for s, d, fill in zip(src, dst, partial):
            whole = self.length[s] // self.page_size
            self.table[d] = self.table[s][:whole]
            copies.append(None)
            if fill:
                self.table[d].append(self.free.pop())
                copies[-1] = (self.table[s][whole], self.table[d][-1], fill)
            self.length[d] = self.length[s]
        return copies

    def rewind(self, lengths: list) -> None:
        for b, r in enumerate(lengths):
            if r >= 0 and r > self.length[b]:
                raise ValueError("past the written length")
            if 0 <= r < self.length[b] and r % self.page_size and self.holders(self.table[b][r // self.page_size]) > 1:
                raise ValueError("into a page that others hold")
        for b in range(len(lengths) - 1, -1, -1):
            if lengths[b] >= 0:
                self._drop(b, pages_for(lengths[b], self.page_size))
                self.length[b] = lengths[b]

    def reset(self, b: int) -> None:
        self._drop(b, 0)
        self.length[b] = 0

    def _drop(self, b: int, keep: int) -> None:
        while len(self.table[b]) > keep:
            page = self.table[b].pop()
            if self.holders(page) == 0:
                self.free.append(page)


def scores(q, k, pos, window=0, cap=0.0, slope=0.0):
    """Scores [rows, keys] of rows q [rows, D] at positions pos over keys k [keys, D] at 0, 1, ..; -inf where not seen."""
    t = np.arange(len(k))[None]
    p = np.asarray(pos)[:, None]
    seen = (t <= p) & ((t > p - window) if window else True)
    with np.errstate(invalid="ignore", over="ignore"):
        z = (q @ np.where(seen.any(0)[:, None], k, 0.0).T) / np.sqrt(q.shape[-1])
        if cap > 0:
            z = cap * np.tanh(z / cap)
        z = z - slope * (p - t)
    return np.where(seen, z, -np.inf)


def attend(z, v):
    """Softmax of scores z [rows, keys] times v [keys, D]; what a row does not see does not count, whatever it holds."""
    w = np.exp(z - z.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        return np.stack([w[i, s] @ v[s] for i, s in enumerate(z > -np.inf)])


def kept_tokens(x, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """Indexes of the kept tokens of a row of logits, in order, and their weights over the largest."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, dtype=np.float64)) + 0.0
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    if not len(order):
        return order, np.zeros(0)
    if not temperature > 0:
        return order[:1], np.ones(1)
    y = x[order]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(y == y[0], 1.0, np.exp((y - y[0]) / float(temperature)))
    n = len(order)
    if top_k > 0:
        n = min(n, int(top_k))
    if top_p < 1:
        total = w[:n].sum()
        before = np.concatenate([[0.0], np.cumsum(w[:n])[:-1]])
        n = int((before < float(top_p) * total).sum())
    if min_p > 0:
        n = min(n, int((w >= float(min_p)).sum()))
    n = max(n, 1)
    return order[:n], w[:n]


def draw_kept(tokens, weights, noise):
    """The token of the largest weight over noise, the lowest of equal ones."""
    if not len(tokens):
        return 0
    race = weights / np.asarray(noise, dtype=np.float64)[tokens]
    return int(tokens[race == race.max()].min())
