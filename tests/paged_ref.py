"""A paged cache kept by plain Python, one step after another, for the GPU tests to compare with."""
from __future__ import annotations

import random

import torch


class RefCache:
    """Books (table, lens, ref) as Python lists and pages as CPU tensors."""

    def __init__(self, rows, cols, n_pages, page, h_kv, d_qk, d_v, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.P, self.cols = page, cols
        self.table = [[-1] * cols for _ in range(rows)]
        self.lens, self.ref = [0] * rows, [0] * n_pages
        # what a page holds before it is written must never matter: NaN
        self.k = torch.full((n_pages, h_kv, page, d_qk), float("nan"), dtype=torch.bfloat16)
        self.v = torch.full((n_pages, h_kv, page, d_v), float("nan"), dtype=torch.bfloat16)
        self.g = g

    def pages_of(self, n):
        return -(-n // self.P)

    def new_tokens(self, rows, most):
        h = self.k.shape[1]
        r = lambda d: torch.randn(rows, h, most, d, generator=self.g).to(torch.bfloat16)  # noqa: E731
        return r(self.k.shape[3]), r(self.v.shape[3])

    def append(self, k_new, v_new, n_new):
        """Returns short_pages; nothing changes unless it is 0."""
        table, lens, ref = [list(r) for r in self.table], list(self.lens), list(self.ref)
        copies, writes, short = [], [], 0
        free = [p for p, n in enumerate(ref) if n <= 0]
        at = 0
        over = any(self.pages_of(n + m) > self.cols for n, m in zip(lens, n_new))
        for b, m in enumerate(n_new):
            if m <= 0:
                continue
            n = lens[b]
            if n % self.P and ref[table[b][n // self.P]] > 1:
                at += 1
                if at <= len(free):
                    old, new = table[b][n // self.P], free[at - 1]
                    copies.append((old, new, n % self.P))
                    ref[old] -= 1
                    ref[new], table[b][n // self.P] = 1, new
                else:
                    ref[table[b][n // self.P]] -= 1
            for c in range(self.pages_of(n), self.pages_of(n + m)):
                at += 1
                if at <= len(free) and c < self.cols:
                    ref[free[at - 1]], table[b][c] = 1, free[at - 1]
            lens[b] = n + m
            writes.append((b, n, m))
        short = max(0, at - len(free))
        if over:
            return -1
        if short:
            return short
        self.table, self.lens, self.ref = table, lens, ref
        for old, new, rows in copies:
            self.k[new, :, :rows], self.v[new, :, :rows] = self.k[old, :, :rows], self.v[old, :, :rows]
        for b, n, m in writes:
            for i in range(m):
                page, row = table[b][(n + i) // self.P], (n + i) % self.P
                self.k[page, :, row], self.v[page, :, row] = k_new[b, :, i], v_new[b, :, i]
        return 0

    def fork(self, src, dst):
        done = []
        start = list(self.lens)
        for i, (a, b) in enumerate(zip(src, dst)):
            ok = 0 <= a < len(self.lens) and 0 <= b < len(self.lens) and start[b] == 0
            ok = ok and b not in dst[:i] and a not in dst
            done.append(int(ok))
            if ok:
                self.table[b], self.lens[b] = list(self.table[a]), self.lens[a]
                for p in self.table[a][:self.pages_of(self.lens[a])]:
                    self.ref[p] += 1
                self.table[b][self.pages_of(self.lens[a]):] = [-1] * (self.cols - self.pages_of(self.lens[a]))
        return done

    def free(self, rows, keep=None):
        done = []
        for i, b in enumerate(rows):
            ok = 0 <= b < len(self.lens) and b not in rows[:i]
            done.append(int(ok))
            if not ok:
                continue
            n = self.lens[b]
            want = 0 if keep is None else keep[i]
            now = n if want < 0 or want > n else want
            for c in range(self.pages_of(now), self.pages_of(n)):
                self.ref[self.table[b][c]] -= 1
                self.table[b][c] = -1
            self.lens[b] = now
        return done

    def compact(self):
        """Returns (remap, n_live)."""
        n_live = sum(n > 0 for n in self.ref)
        holes = [p for p, n in enumerate(self.ref) if n <= 0 and p < n_live]
        movers = [p for p, n in enumerate(self.ref) if n > 0 and p >= n_live]
        remap = [p if n > 0 else -1 for p, n in enumerate(self.ref)]
        for f, t in zip(movers, holes):
            remap[f] = t
            self.k[t], self.v[t] = self.k[f], self.v[f]
            self.ref[t], self.ref[f] = self.ref[f], 0
        for b, n in enumerate(self.lens):
            for c in range(self.pages_of(n)):
                self.table[b][c] = remap[self.table[b][c]]
        return remap, n_live

    def dense(self, b):
        """(k [Hkv, n, d], v) of row b."""
        n = self.lens[b]
        pages = self.table[b][:self.pages_of(n)]
        cut = lambda x: x[pages].transpose(0, 1).flatten(1, 2)[:, :n]  # noqa: E731
        return cut(self.k), cut(self.v)

    def on_gpu(self):
        i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(k_pages=self.k.cuda(), v_pages=self.v.cuda(), table=i(self.table), lens=i(self.lens),
                    ref=i(self.ref))

    def assert_equal(self, x, what=""):
        assert x["table"].tolist() == self.table, what + " table"
        assert x["lens"].tolist() == self.lens, what + " lens"
        assert x["ref"].tolist() == self.ref, what + " ref"
        assert torch.equal(x["k_pages"].cpu().view(torch.int16), self.k.view(torch.int16)), what + " k"
        assert torch.equal(x["v_pages"].cpu().view(torch.int16), self.v.view(torch.int16)), what + " v"


def filled(rows, cols, n_pages, page, h_kv, d_qk, d_v, lens, seed=0):
    """A cache whose rows have the given lengths, on pages handed out in a shuffled order."""
    c = RefCache(rows, cols, n_pages, page, h_kv, d_qk, d_v, seed)
    order = list(range(n_pages))
    random.Random(seed).shuffle(order)
    for b, n in enumerate(lens):
        for col in range(c.pages_of(n)):
            p = order.pop()
            c.table[b][col], c.ref[p] = p, 1
            m = min(c.P, n - col * c.P)
            c.k[p, :, :m] = torch.randn(h_kv, m, d_qk, generator=c.g).to(torch.bfloat16)
            c.v[p, :, :m] = torch.randn(h_kv, m, d_v, generator=c.g).to(torch.bfloat16)
        c.lens[b] = n
    return c
