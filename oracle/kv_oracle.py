"""Plain CPU definition (NumPy, fp64) of the paged key-value cache and of the
attention over it: what the kernels behind include/qgkv.h have to give.

Page by page and token by token, in Python loops: it defines the results, it is
not meant to be fast.  It shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np

SHORT, LONG, PAIR = 1, 2, 4


def sees(pos: int, t: int, window: int, sinks: int) -> bool:
    """Does the row at position pos see token t?"""
    return 0 <= t <= pos and (window == 0 or t > pos - window or t < sinks)


def attend_row(q, k, v, pos: int, scale: float, window: int = 0, sinks: int = 0) -> np.ndarray:
    """One row: q [D], k and v [tokens][D]; 0 where the row sees nothing."""
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    t = np.array([i for i in range(k.shape[0]) if sees(pos, i, window, sinks)], dtype=np.int64)
    if t.size == 0:
        return np.zeros(v.shape[1])
    with np.errstate(all="ignore"):
        s = scale * (k[t] @ q)
        w = np.exp(s - s.max())
        return (w / w.sum()) @ v[t]


class Cache:
    """pool [pages][layers][2][kv_heads][page_size][head_dim], tables, lens, refs."""

    def __init__(self, pool, tables, lens, refs):
        self.pool, self.tables = np.array(pool), np.array(tables)
        self.lens, self.refs = np.array(lens), np.array(refs)
        self.info = [0, 0, 0, 0]
        self.refused = 0  # the bit that the last extend was refused with
        self.P = self.pool.shape[4]

    def used(self, s: int, length=None) -> int:
        n = int(self.lens[s]) if length is None else int(length)
        return -(-n // self.P)

    def tokens(self, s: int, layer: int, which: int) -> np.ndarray:
        """[tokens][kv_heads][head_dim] of a slot."""
        n = int(self.lens[s])
        pages = [self.pool[self.tables[s, i], layer, which] for i in range(self.used(s))]
        if not pages:
            return np.zeros((0,) + self.pool.shape[3:4] + self.pool.shape[5:], dtype=self.pool.dtype)
        return np.concatenate([p.transpose(1, 0, 2) for p in pages])[:n]

    def append(self, layer: int, slots, rows, k, v, max_rows=None):
        if self.refused & self.info[0]:
            return
        at = 0
        for s, r in zip(slots, rows):
            for i in range(r if max_rows is None else min(r, max_rows)):
                pos = int(self.lens[s]) - r + i
                if pos >= 0:
                    page = self.tables[s, pos // self.P]
                    self.pool[page, layer, 0, :, pos % self.P] = k[at + i]
                    self.pool[page, layer, 1, :, pos % self.P] = v[at + i]
            at += r

    def attend(self, layer: int, slots, rows, q, scale: float, window: int = 0, sinks: int = 0) -> np.ndarray:
        out, at = np.zeros(q.shape), 0
        group = q.shape[1] // self.pool.shape[3]
        for s, r in zip(slots, rows):
            k, v = (self.tokens(s, layer, w).astype(np.float64) for w in (0, 1))
            for i in range(r):
                for h in range(q.shape[1]):
                    out[at + i, h] = attend_row(q[at + i, h], k[:, h // group], v[:, h // group],
                                                int(self.lens[s]) - r + i, scale, window, sinks)
            at += r
        return out

    def extend(self, n_new):
        n_new = [max(int(n), 0) for n in n_new]
        slots = range(len(self.lens))
        if any(int(self.lens[s]) + n_new[s] > self.tables.shape[1] * self.P for s in slots):
            self.info[0] |= LONG
            self.refused = LONG
            return
        # slots that would write into a page that others name too
        tail = {s: int(self.tables[s, self.used(s) - 1]) for s in slots if n_new[s] > 0 and self.lens[s] % self.P != 0}
        shared = {s: p for s, p in tail.items() if self.refs[p] > 1}
        copies = []
        for s, p in shared.items():
            growing = [x for x, y in shared.items() if y == p]
            if not (len(growing) == self.refs[p] and min(growing) == s):
                copies.append(s)
        need = {s: self.used(s, int(self.lens[s]) + n_new[s]) - self.used(s) for s in slots}
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        total = sum(need.values()) + len(copies)
        if total > len(free):
            self.info[0] |= SHORT
            self.info[1] = total - len(free)
            self.refused = SHORT
            return
        self.refused = 0
        for s in slots:
            if s in copies:
                p = free.pop(0)
                self.pool[p] = self.pool[shared[s]]
                self.refs[p] = 1
                self.tables[s, self.used(s) - 1] = p
            for i in range(need[s]):
                p = free.pop(0)
                self.refs[p] = 1
                self.tables[s, self.used(s) + i] = p
        for s in copies:
            self.refs[shared[s]] -= 1
        for s in slots:
            self.lens[s] += n_new[s]

    def fork(self, src, dst):
        lens, n = self.lens.copy(), len(self.lens)
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < n and 0 <= d < n) or lens[d] != 0 or d in dst[:i] or s in dst:
                self.info[0] |= PAIR
                continue
            u = self.used(s)
            self.tables[d, :u] = self.tables[s, :u]
            for p in self.tables[s, :u]:
                self.refs[p] += 1
            self.lens[d] = self.lens[s]

    def trim(self, seqs, keep=None):
        for i, s in enumerate(seqs):
            if not 0 <= s < len(self.lens) or s in seqs[:i]:
                self.info[0] |= PAIR
                continue
            left = min(max(int(keep[i]), 0), int(self.lens[s])) if keep is not None else 0
            for j in range(self.used(s, left), self.used(s)):
                self.refs[self.tables[s, j]] -= 1
                self.tables[s, j] = -1
            self.lens[s] = left

    def compact(self):
        live = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        m = len(live)
        moves = list(zip([p for p in live if p >= m], [p for p in range(m) if self.refs[p] == 0]))
        for a, b in moves:
            self.pool[b] = self.pool[a]
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.tables[self.tables == a] = b
        self.info[2:] = [m, len(moves)]
