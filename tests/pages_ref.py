"""Plain references of the page operators, on lists and numpy arrays: what
include/fp8pa.h says, one row and one page at a time."""
import numpy as np

BLOCK, LEN, OFFSETS, TREE, ROW, NO_BLOCK, SHARED = 2, 4, 32, 64, 128, 256, 512


class Pool:
    """Tables, lengths and counts of rows over `nb` pages, and arrays of pages."""

    def __init__(self, rows, cols, nb, bs, arrays=()):
        self.t = np.full((rows, cols), -1, np.int32)
        self.n = np.zeros(rows, np.int32)
        self.r = np.zeros(nb, np.int32)
        self.nb, self.bs, self.arrays, self.flags = nb, bs, list(arrays), 0

    def good(self, n):
        return 0 <= n <= self.t.shape[1] * self.bs

    def pages(self, n):
        return -(-int(n) // self.bs)

    def free(self):
        return [int(p) for p in np.flatnonzero(self.r == 0)]

    def fill(self, rng, lens):
        """Rows of these lengths on pages in a random order."""
        order = list(rng.permutation(self.nb))
        for b, n in enumerate(lens):
            self.n[b] = n
            for c in range(self.pages(n)):
                self.t[b, c] = order.pop()
                self.r[self.t[b, c]] = 1
        return self

    def keep(self, accepted, offsets):
        new = self.n.copy()
        for b, path in enumerate(accepted):
            lo, hi, n = int(offsets[b]), int(offsets[b + 1]), int(self.n[b])
            if lo < 0 or hi < lo:
                self.flags |= OFFSETS
                continue
            if not self.good(n) or n < hi - lo:
                self.flags |= LEN
                continue
            kept = []
            for a in path:
                if a < 0:
                    break
                if a >= hi - lo or (kept and a <= kept[-1]):
                    self.flags |= TREE
                    break
                kept.append(int(a))
            ctx = n - (hi - lo)
            new[b] = ctx + len(kept)
            for t, a in enumerate(kept):
                if a == t:
                    continue
                src, dst = ctx + a, ctx + t
                p, q = self.t[b, src // self.bs], self.t[b, dst // self.bs]
                if not (0 <= p < self.nb and 0 <= q < self.nb):
                    self.flags |= BLOCK
                    continue
                for x in self.arrays:
                    x[q, :, dst % self.bs] = x[p, :, src % self.bs]
        return new

    def fork(self, src, dst):
        rows = self.t.shape[0]
        n0, t0 = self.n.copy(), self.t.copy()
        free, made = self.free(), set()
        for s, d in zip(src, dst):
            first = d not in made
            if 0 <= d < rows:
                made.add(d)
            if not (0 <= s < rows and 0 <= d < rows) or s == d or n0[d] != 0 or not first:
                self.flags |= ROW
                continue
            n = int(n0[s])
            if not self.good(n):
                self.flags |= LEN
                continue
            last = -1
            if n % self.bs:
                old = t0[s, n // self.bs]
                if not 0 <= old < self.nb:
                    self.flags |= BLOCK
                    continue
                if not free:
                    self.flags |= NO_BLOCK
                    continue
                last = free.pop(0)
                for x in self.arrays:
                    x[last] = x[old]
            self.n[d] = n
            for c in range(self.t.shape[1]):
                p = -1
                if c < self.pages(n):
                    p = last if c == n // self.bs else int(t0[s, c])
                    if 0 <= p < self.nb:
                        self.r[p] += 1
                    else:
                        self.flags |= BLOCK
                self.t[d, c] = p

    def resize(self, then):
        r0, left = self.r.copy(), set()
        for b, m in enumerate(then):
            n, m = int(self.n[b]), int(m)
            if not self.good(n) or not self.good(m):
                self.flags |= LEN
                left.add(b)
                continue
            k = min(n, m)
            if n != m and k % self.bs:
                p = self.t[b, k // self.bs]
                if 0 <= p < self.nb and r0[p] > 1:
                    self.flags |= SHARED
                    left.add(b)
        for b, m in enumerate(then):
            if b in left:
                continue
            for c in range(self.pages(m), self.pages(self.n[b])):
                p = self.t[b, c]
                if 0 <= p < self.nb:
                    self.r[p] -= 1
                else:
                    self.flags |= BLOCK
                self.t[b, c] = -1
        free, want = self.free(), 0
        for b, m in enumerate(then):
            if b in left:
                continue
            old, new = self.pages(self.n[b]), self.pages(m)
            if new > old:
                want += new - old
                if want > len(free):
                    self.flags |= NO_BLOCK
                    continue
                for c in range(old, new):
                    self.t[b, c] = free[want - (new - c)]
                    self.r[self.t[b, c]] = 1
            self.n[b] = m

    def compact(self):
        live = int((self.r > 0).sum())
        low = [p for p in self.free() if p < live]
        high = [p for p in range(live, self.nb) if self.r[p] > 0]
        to = np.where(self.r > 0, np.arange(self.nb), -1).astype(np.int32)
        for h, lo in zip(high, low):
            to[h] = lo
            for x in self.arrays:
                x[lo] = x[h]
            self.r[lo], self.r[h] = self.r[h], 0
        for b, n in enumerate(self.n):
            if not self.good(n):
                self.flags |= LEN
                continue
            for c in range(self.pages(n)):
                p = self.t[b, c]
                if 0 <= p < self.nb and to[p] >= 0:
                    self.t[b, c] = to[p]
                else:
                    self.flags |= BLOCK
        return to
