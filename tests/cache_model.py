"""A plain model of the paged cache and of attention over it, for the tests:
lists and dictionaries, one row at a time, and attention in 64 bits."""
import math

import numpy as np


class CacheModel:
    """What the cache calls are to do: tables, lengths, holders, and which
    token's row lies at (page, row)."""

    def __init__(self, slots, max_pages, pages, P):
        self.P, self.max_pages = P, max_pages
        self.table = [[] for _ in range(slots)]
        self.len = [0] * slots
        self.refs = [0] * pages
        self.rows = {}  # (page, row) -> mark

    def _take(self):
        p = self.refs.index(0)
        self.refs[p] = 1
        return p

    def grow(self, slots, counts):
        """Returns the batch positions that failed."""
        free, before, failed, todo = self.refs.count(0), 0, [], []
        for b, (s, c) in enumerate(zip(slots, counts)):
            new = self.len[s] + c
            if c < 0 or -(-new // self.P) > self.max_pages:
                failed.append(b)
                continue
            need = -(-new // self.P) - len(self.table[s])
            before += need
            if need and before > free:
                failed.append(b)
                continue
            todo.append((s, need, new))
        for s, need, new in todo:
            self.table[s] += [self._take() for _ in range(need)]
            self.len[s] = new
        return failed

    def append(self, slots, marks):
        """marks[b]: the rows for the last len(marks[b]) positions."""
        for s, m in zip(slots, marks):
            for i, x in enumerate(m):
                pos = self.len[s] - len(m) + i
                self.rows[self.table[s][pos // self.P], pos % self.P] = x

    def fork(self, src, dst):
        free, before, failed, todo = self.refs.count(0), 0, [], []
        for b, (s, d) in enumerate(zip(src, dst)):
            if s == d or self.len[d]:
                failed.append(b)
                continue
            part = self.len[s] % self.P
            before += part > 0
            if part and before > free:
                failed.append(b)
                continue
            todo.append((s, d, part))
        tails = [self._take() if part else None for _, _, part in todo]
        for (s, d, part), tail in zip(todo, tails):
            whole = self.table[s][:self.len[s] // self.P]
            for p in whole:
                self.refs[p] += 1
            self.table[d] = list(whole)
            self.len[d] = self.len[s]
            if part:
                self.table[d].append(tail)
                for r in range(part):
                    if (self.table[s][-1], r) in self.rows:
                        self.rows[tail, r] = self.rows[self.table[s][-1], r]
        return failed

    def free(self, slots):
        for s in slots:
            for p in self.table[s]:
                self.refs[p] -= 1
            self.table[s], self.len[s] = [], 0

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        src = [p for p, r in enumerate(self.refs) if r and p >= live]
        dst = [p for p, r in enumerate(self.refs) if not r and p < live]
        to = dict(zip(src, dst))
        for s, t in enumerate(self.table):
            for i, p in enumerate(t):
                if p in to:
                    for r in range(min(self.P, self.len[s] - i * self.P)):
                        if (p, r) in self.rows:
                            self.rows[to[p], r] = self.rows[p, r]
            self.table[s] = [to.get(p, p) for p in t]
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        return len(src)


def random_tree(rng, N, wide=3):
    return [-1] + [int(max(0, i - 1 - rng.integers(0, wide))) for i in range(1, N)]


def masks_of(parent, nodes, N):
    out = []
    for n in range(N):
        m = 0
        if n < nodes:
            a = n
            while a >= 0:
                m |= 1 << int(a)
                p = parent[a] if a > 0 else -1
                a = p if 0 <= p < a else -1
        out.append(m)
    return out


def accept_of(tok, parent, nodes, argmax):
    """The accepted path, node by node."""
    path = [0] if nodes > 0 else []
    while path:
        at = path[-1]
        nxt = [n for n in range(1, nodes) if parent[n] == at and at < n and tok[n] >= 0 and tok[n] == argmax[at]]
        if not nxt:
            break
        path.append(nxt[0])
    return path


def attend_row(q, keys, vals, scale):
    """One row in 64 bits over the keys it sees: (output, sum of p |v|)."""
    if len(keys) == 0:
        z = np.zeros(vals.shape[1])
        return z, z
    s = keys @ q * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ vals, p @ np.abs(vals)


# Half a unit in the last place, relative, of a value rounded to the type.
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def tolerance(kind, ref, size, keys, vmax):
    """How far an output may be from 64 bits.  Each weight p is rounded once
    (relative UNIT), the result once more; scores and sums are float32, whose
    errors (a sum of at most 256 products, exp, a running sum) stay below
    2^-14 of the sum of p |v| at the tests' magnitudes.  float16 weights
    below 2^-14 of the largest's 2^7 are rounded to multiples of 2^-24, half
    of which over the largest is 2^-32 each; a float16 output below 2^-14 to
    multiples of 2^-24."""
    u = UNIT[kind]
    tol = u * np.abs(ref) + (u + 2.0 ** -14) * size
    if kind == "f16":
        tol = tol + keys * 2.0 ** -32 * vmax + 2.0 ** -24
    return tol + 1e-30


def scaled(x):
    return x / math.sqrt(x.shape[-1])
