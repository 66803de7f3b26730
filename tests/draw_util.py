"""The draw from a filter set, the verification of drafts and the pages of a
cache, from their definitions in 64 bits (NumPy, one row or request at a time).
"""
from __future__ import annotations

import math

import numpy as np

# An index or a set may differ from the definition's where a border lies this
# close (relative to the row's mass): every weight is off by at most 2^-39 of
# itself and half a unit 2^-44, and a row's mass is at least one weight of 1.
def tolerance(V):
    return 2.0 ** -38 + V * 2.0 ** -44


def filter_set(x, T, k=0, p=1.0, m=0.0):
    """(weights, gap) of one row: exp((x - M) / T) inside the set and 0 outside
    (None: no candidate), and how close a filter's border is to a neighbouring
    element. Greedy rows and rows with +inf have one weight."""
    x = np.asarray(x, np.float32).astype(np.float64)
    cand = x > -np.inf
    if not cand.any():
        return None, np.inf
    top = x[cand].max()
    w = np.zeros(x.size)
    T = float(np.float32(T))
    if not T > 0 or top == np.inf:
        w[np.flatnonzero(cand & (x == top))[0]] = 1
        return w, np.inf
    T = max(T, 2.0 ** -126)
    ids = np.flatnonzero(cand)
    ids = ids[np.argsort(-x[ids], kind="stable")]
    with np.errstate(over="ignore"):
        z = (x[ids] - top) / T
    e = np.exp(z)
    many, gap = len(ids), np.inf
    if k >= 1:
        many = min(many, int(k))
    p, m = float(np.float32(p)), float(np.float32(m))
    if p <= 0:
        many = 1
    elif p < 1:
        c = np.cumsum(e)
        n = int(np.searchsorted(c, p * c[-1], "left")) + 1
        many = min(many, n)
        gap = np.abs(c - p * c[-1]).min() / c[-1]
    if m > 0:
        border = math.log(min(m, 1.0))
        n = int(np.count_nonzero(z >= border))
        many = min(many, n)
        if 0 < m < 1:
            gap = min(gap, np.abs(z - border).min() * 1e3)  # borders in 64 bits on both sides
    many = max(many, 1)
    w[ids[:many]] = e[:many]
    return w, gap


def pick(w, u):
    """(index, gap): the smallest index whose cumulative weight passes u of the
    total, and the distance of that point from the nearest boundary."""
    u = float(np.float32(u))
    u = 0.0 if not u > 0 else min(u, 1 - 2.0 ** -24)
    c = np.cumsum(w)
    t = u * c[-1]
    i = int(np.searchsorted(c, t, "right"))
    gap = min(abs(c[i] - t), abs(t - (c[i - 1] if i else -np.inf))) / c[-1]
    return i, gap


def draw(x, T, u, k=0, p=1.0, m=0.0):
    """(index, logprob, gap) of one row."""
    w, gap = filter_set(x, T, k, p, m)
    if w is None:
        return -1, -np.inf, np.inf
    if np.count_nonzero(w) == 1:
        return int(np.flatnonzero(w)[0]), 0.0, gap
    i, g = pick(w, u)
    return i, math.log(w[i] / w.sum()), min(gap, g)


def verify(x, draft, offsets, T, u, u_draw, q=None, k=None, p=None, m=None):
    """(tokens, count, gaps): tokens int64 [R] with -2 in rows of no request,
    and per request how close a decision was."""
    R = len(x)
    out = np.full(R, -2, np.int64)
    n = len(offsets) - 1
    count, gaps = np.zeros(n, np.int32), np.full(n, np.inf)
    for i in range(n):
        r0, r1 = max(0, int(offsets[i])), min(R, int(offsets[i + 1]))
        if r1 <= r0:
            continue
        out[r0:r1] = -1
        for r in range(r0, r1):
            w, gap = filter_set(x[r], T[i], 0 if k is None else k[i], 1.0 if p is None else p[i],
                                0.0 if m is None else m[i])
            gaps[i] = min(gaps[i], gap)
            if w is None:
                break
            w = w / w.sum()
            qr = np.zeros(w.size)
            t = int(draft[r])
            inside = 0 <= t < w.size
            if r + 1 < r1:
                if q is not None:
                    qr = np.nan_to_num(np.asarray(q[r], np.float64), nan=0.0, posinf=1e300)
                    qr = np.maximum(qr, 0)
                elif inside:
                    qr[t] = 1
                uu = float(np.clip(np.nan_to_num(np.float32(u[r])), 0, 1 - 2.0 ** -24))
                if inside and w[t] > 0 and uu * qr[t] < w[t]:
                    if np.count_nonzero(w) > 1:
                        gaps[i] = min(gaps[i], abs(uu * qr[t] - w[t]))
                    out[r] = t
                    count[i] += 1
                    continue
                if inside:
                    gaps[i] = min(gaps[i], abs(uu * qr[t] - w[t]) if w[t] > 0 else np.inf)
            one = np.count_nonzero(w) == 1
            rest = np.maximum(w - np.minimum(qr, 1), 0)
            if one or rest.sum() <= 0:
                rest = w
            out[r], g = pick(rest, u_draw[i])
            if np.count_nonzero(rest) > 1:
                gaps[i] = min(gaps[i], g * rest.sum())
            count[i] += 1
            break
    return out, count, gaps


class Pages:
    """A plain scheduler's page tables."""

    def __init__(self, slots, pages, page, columns):
        self.page, self.columns, self.pages = page, columns, pages
        self.held = [[] for _ in range(slots)]
        self.length = [0] * slots
        self.free = list(range(pages - 1, -1, -1))

    def extend(self, counts, slots):
        start, maps, lengths, tables = [], [], [], []
        left = len(self.free)
        for s, c in zip(slots, counts):
            ok = 0 <= s < len(self.held) and list(slots).count(s) == 1 and \
                self.length[s] + c <= self.columns * self.page
            if ok:
                need = -(-(self.length[s] + c) // self.page) - len(self.held[s])
                left -= need
                ok = need == 0 or left >= 0
            if not ok:
                start.append(-1)
                maps.append([-1] * c)
                lengths.append(0)
                tables.append([])
                continue
            start.append(self.length[s])
            self.held[s] += [self.free.pop() for _ in range(need)]
            maps.append([self.held[s][t // self.page] * self.page + t % self.page
                         for t in range(self.length[s], self.length[s] + c)])
            self.length[s] += c
            lengths.append(self.length[s])
            tables.append(list(self.held[s]))
        return start, maps, lengths, tables

    def trim(self, slots, start, keep):
        """The pages go back so that the same extension takes the same ones."""
        back = []
        for s, a, b in zip(slots, start, keep):
            if not 0 <= s < len(self.held) or list(slots).count(s) > 1 or a < 0:
                continue
            now = max(0, a + b)
            if now >= self.length[s]:
                continue
            n = -(-now // self.page)
            back += self.held[s][n:]
            self.held[s] = self.held[s][:n]
            self.length[s] = now
        self.free += back[::-1]

    def table(self):
        return np.array([h + [-1] * (self.columns - len(h)) for h in self.held], np.int32)
