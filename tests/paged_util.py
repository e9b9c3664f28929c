"""Plain implementations for the paged cache's tests: its bookkeeping row by row and page by page on lists, and the
chunk attention in 64 bits, with the error bound that the kernels' roundings allow."""
import math

import torch

CAPACITY, LENGTH, NODE, PAGE, ROW = 4, 8, 2, 32, 64


class Book:
    """refs, length, held and table of a cache, on lists; each call returns the error bits it raises."""

    def __init__(self, rows, max_pages, num_pages, ps):
        self.rows, self.max_pages, self.num_pages, self.ps = rows, max_pages, num_pages, ps
        self.refs = [0] * num_pages
        self.length, self.held = [0] * rows, [0] * rows
        self.table = [[-1] * max_pages for _ in range(rows)]

    def need(self, tokens):
        return -(-tokens // self.ps)

    def free(self, keep):
        for r, k in enumerate(keep):
            if k < 0:
                continue
            self.length[r] = min(self.length[r], k)
            for c in range(self.need(self.length[r]), self.held[r]):
                self.refs[self.table[r][c]] -= 1
                self.table[r][c] = -1
            self.held[r] = self.need(self.length[r])
        return 0

    def fork(self, src, dst):
        err, empty = 0, [ln == 0 and h == 0 for ln, h in zip(self.length, self.held)]
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < self.rows and 0 <= d < self.rows) or d in dst[:i] or s in dst or d in src or not empty[d]:
                err |= ROW
                continue
            self.length[d], self.held[d] = self.length[s], self.need(self.length[s])
            for c in range(self.held[d]):
                self.table[d][c] = self.table[s][c]
                self.refs[self.table[s][c]] += 1
        return err

    def reserve(self, n_new):
        """(copies, granted, err)"""
        err, copies, granted, short = 0, [], [], False
        free = [p for p, x in enumerate(self.refs) if x == 0]
        for r, n in enumerate(n_new):
            end = self.length[r] + n
            bad = LENGTH if n < 0 else CAPACITY if end > self.max_pages * self.ps else 0
            if bad:
                err |= bad
                granted.append(0)
                continue
            t = self.length[r] // self.ps
            cow = n > 0 and self.length[r] % self.ps != 0 and self.refs[self.table[r][t]] > 1
            more = max(0, self.need(end) - self.held[r]) if n > 0 else 0
            short = short or more + cow > len(free)
            granted.append(0 if short else 1)
            if short:
                err |= CAPACITY if n > 0 else 0
                continue
            if cow:
                p = free.pop(0)
                self.refs[self.table[r][t]] -= 1
                copies.append([self.table[r][t], p, self.length[r] % self.ps, r])
                self.table[r][t], self.refs[p] = p, 1
            for _ in range(more):
                p = free.pop(0)
                self.table[r][self.held[r]], self.refs[p] = p, 1
                self.held[r] += 1
        return copies, granted, err

    def commit(self, rows, n_new, bias):
        err, done = 0, set()
        for r, n in zip(rows, n_new):
            if not 0 <= r < self.rows or r in done:
                err |= ROW
                continue
            done.add(r)
            if n < 0:
                err |= LENGTH
            elif self.length[r] + n + bias > self.held[r] * self.ps:
                err |= CAPACITY
            else:
                self.length[r] += n + bias
        return err

    def compact(self):
        n = sum(x > 0 for x in self.refs)
        out = [p for p in range(n, self.num_pages) if self.refs[p]]
        goes = dict(zip(out, [p for p in range(n) if not self.refs[p]]))
        for a, z in goes.items():
            self.refs[z], self.refs[a] = self.refs[a], 0
        self.table = [[goes.get(p, p) for p in row] for row in self.table]
        return [[a, z, self.ps, -1] for a, z in goes.items()]

    def state(self):
        words = [sum((self.refs[w * 32 + k] == 0) << k for k in range(min(32, self.num_pages - w * 32)))
                 for w in range(-(-self.num_pages // 32))]
        words = [w - 2 ** 32 if w >= 2 ** 31 else w for w in words]
        return torch.tensor(self.refs + words + self.length + self.held + sum(self.table, []), dtype=torch.int32)

    def check(self):
        """refs count the holders."""
        held = [p for r in range(self.rows) for p in self.table[r][:self.held[r]]]
        assert [held.count(p) for p in range(self.num_pages)] == self.refs

    def slots(self, r, x):
        """(page, line) tensors of row r's tokens x (a tensor)."""
        tab = torch.tensor(self.table[r], device=x.device)
        return tab[x // self.ps], x % self.ps


def rotate(x, pos, theta):
    """x [n][heads][D] float64, pos [n]: pairs (j, j + D/2) by pos * theta^(-2j/D)."""
    D = x.shape[-1]
    freq = torch.tensor([float(theta) ** (-2.0 * j / D) for j in range(D // 2)], dtype=torch.float64, device=x.device)
    ang = (pos.double()[:, None] * freq)[:, None]
    lo, hi = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([lo * ang.cos() - hi * ang.sin(), hi * ang.cos() + lo * ang.sin()], -1)


def attention(q, k, v, seen, scale, half_step, terms):
    """One head, 64 bits: q [n][D] rotated, k, v [x][D], seen [n][x].  Returns the output and the error the kernels may
    make: with u = half_step, a score is off by at most e = (u + terms 2^-24) scale sum |q_j k_j| (q rounded once, the
    products summed in 32 bits), so a weight by e plus u for its own rounding and terms 2^-24 for the sums, and the
    normaliser by the mean of e; then the result is rounded.  First order, times 1.2 for the higher ones."""
    z = (q @ k.T * scale).masked_fill(~seen, -math.inf)
    any_key = seen.any(1, keepdim=True)
    p = torch.where(any_key, torch.softmax(z.masked_fill(~any_key, 0.0), -1), torch.zeros_like(z))
    out = p @ v
    w = terms * 2.0 ** -24
    e = (half_step + w) * scale * (q.abs() @ k.abs().T)
    mean = (p * e).sum(1, keepdim=True)
    tol = 1.2 * ((p * (e + mean + half_step + w)) @ v.abs()) + half_step * out.abs() + 1e-30
    return out, tol


def half_step(dtype):
    return torch.finfo(dtype).eps / 2
