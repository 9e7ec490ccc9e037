"""Plain restatements, in 64 bits and in Python loops, of the paged 4-bit
cache (include/dspark_kv4.h): the format, attention over it, and the pages'
bookkeeping.  Test infrastructure only."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    """The 256 E4M3 bytes as the cache reads them (a NaN is 448)."""
    out = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            out[b] = 448.0
            continue
        out[b] = -v if b & 128 else v
    return out


E4M3 = e4m3_values()
POSITIVE = E4M3[:127]  # ascending, byte == index


def nearest(grid, x):
    """Index of the nearest of an ascending grid, ties to the even index."""
    i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo, hi = grid[i - 1], grid[i]
    d0, d1 = x - lo, hi - x
    low = (d0 < d1) | ((d0 == d1) & ((i - 1) % 2 == 0))
    return np.where(x >= grid[-1], len(grid) - 1, np.where(low, i - 1, i))


def quantise(x, g):
    """x float64 [..., 16 n], g broadcastable: codes (uint8), scales (uint8)."""
    y = np.asarray(x, np.float64) / g
    y = np.where(np.isnan(y), 0.0, y).reshape(*x.shape[:-1], -1, 16)
    top = np.abs(y).max(-1)
    scale = nearest(POSITIVE, np.minimum(top / 6, 448.0)).astype(np.uint8)
    s = POSITIVE[scale][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        a = np.where(s > 0, np.minimum(np.abs(y) / s, 6.0), 0.0)
    code = nearest(E2M1, a) + 8 * (y < 0)
    return code.astype(np.uint8).reshape(x.shape), scale


def values(code, scale, g):
    """What codes [..., 16 n] and scales [..., n] stand for."""
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    v = v.reshape(*code.shape[:-1], -1, 16) * E4M3[scale][..., None]
    return v.reshape(code.shape) * g


class Cache:
    """A cache's bytes on the host: data uint8 [num_pages, page bytes]."""

    def __init__(self, num_pages, page, heads, dim, gk=None, gv=None, rng=None):
        self.page, self.heads, self.dim, self.num_pages = page, heads, dim, num_pages
        self.record = page * (dim + dim // 8)
        rng = rng or np.random.default_rng(0)
        self.data = rng.integers(0, 256, (num_pages, heads * self.record), dtype=np.uint8)
        one = np.ones(heads)
        self.g = (one if gk is None else np.asarray(gk, np.float64), one if gv is None else np.asarray(gv, np.float64))

    def sections(self, page, head):
        r = self.data[page, head * self.record:(head + 1) * self.record]
        half, eighth = self.page * self.dim // 2, self.page * self.dim // 16
        codes = [r[i * half:(i + 1) * half].reshape(self.page, -1) for i in range(2)]
        scales = [r[2 * half + i * eighth:2 * half + (i + 1) * eighth].reshape(self.page, -1) for i in range(2)]
        return codes, scales

    def store(self, page, row, k, v):
        """k, v float64 [heads, dim] into a page's row."""
        for h in range(self.heads):
            codes, scales = self.sections(page, h)
            for w, x in enumerate((k, v)):
                c, s = quantise(x[h], self.g[w][h])
                codes[w][row] = c[0::2] | (c[1::2] << 4)
                scales[w][row] = s

    def load(self, page, row, head):
        codes, scales = self.sections(page, head)
        out = []
        for w in range(2):
            b = codes[w][row]
            c = np.stack([b & 15, b >> 4], -1).reshape(-1)
            out.append(values(c, scales[w][row], self.g[w][head]))
        return out

    def tokens(self, pages, length, head):
        """k, v [length, dim], and which tokens are there."""
        k, v = np.zeros((length, self.dim)), np.zeros((length, self.dim))
        there = np.zeros(length, bool)
        for t in range(length):
            p = pages[t // self.page]
            if 0 <= p < self.num_pages:
                there[t] = True
                k[t], v[t] = self.load(p, t % self.page, head)
        return k, v, there


def attention(cache, row_start, slots, lens, table, q, group, scale, window):
    """out, lse and, for each output, how far a computation may be from it.

    Bounds, first order, u = 2^-24: a score's FP32 dot product of D exact
    products is off by at most (D + 2) u sum |q k| scale (and the factors'
    three roundings); the maximum's subtraction rounds once more on a number no
    larger than the scores' spread; the exponential is good to 2^-21.  So a weight
    is off by a share d; entering the second product as FP16 adds 2^-11; FP16's
    smallest numbers add 2^-29 of the largest weight.  Sums of n terms in FP32
    add (n / 16 + 16) u at most in the order that the kernels use (16 tokens an
    instruction)."""
    total, qh, dim = q.shape
    out, lse, tol = np.zeros(q.shape), np.full((total, qh), -np.inf), np.zeros(q.shape)
    u = 2.0 ** -24
    for i in range(len(row_start) - 1):
        slot = slots[i]
        n = row_start[i + 1] - row_start[i]
        if n <= 0 or not 0 <= slot < len(lens):
            continue
        length = min(max(int(lens[slot]), 0), table.shape[1] * cache.page)
        for h in range(cache.heads):
            k, v, there = cache.tokens(table[slot], length, h)
            for j in range(n):
                p = length - n + j
                t = np.arange(length)
                seen = there & (t <= p)
                if window:
                    seen &= t > p - window
                if not seen.any():
                    continue
                ks, vs = k[seen], v[seen]
                for m in range(group):
                    row, head = row_start[i] + j, h * group + m
                    x = q[row, head].astype(np.float64)
                    s = ks @ x * scale
                    top = s.max()
                    w = np.exp(s - top)
                    y = (w @ vs) / w.sum()
                    out[row, head], lse[row, head] = y, top + np.log(w.sum())
                    d = (dim + 6) * u * (np.abs(ks) @ np.abs(x) * abs(scale)).max() + 2.0 ** -20
                    d += 4 * u * np.abs(s - top).max() + (len(s) / 16 + 16) * u
                    size = (w @ np.abs(vs)) / w.sum()
                    tol[row, head] = (2.0 ** -11 + 2 * d) * size + 2.0 ** -29 * np.abs(vs).sum(0)
    return out, lse, tol


# ---- pages -------------------------------------------------------------------

class Pool:
    def __init__(self, num_pages, page, slots, max_pages):
        self.page, self.max_pages = page, max_pages
        self.refs = np.zeros(num_pages, np.int64)
        self.table = np.full((slots, max_pages), -1, np.int64)
        self.lens = np.zeros(slots, np.int64)

    def up(self, n):
        return -(-int(n) // self.page)

    def there(self, slot):
        return 0 <= slot < len(self.lens)

    def trim(self, slots, new_len):
        for s, n in zip(slots, new_len):
            if not self.there(s) or n < 0 or n >= self.lens[s]:
                continue
            for j in range(self.up(n), self.up(self.lens[s])):
                self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1
            self.lens[s] = n

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            if not self.there(a) or not self.there(b) or a == b:
                continue
            held, now = self.up(self.lens[b]), self.up(self.lens[a])
            for j in range(max(held, now)):
                if j < held:
                    self.refs[self.table[b, j]] -= 1
                self.table[b, j] = self.table[a, j] if j < now else -1
                if j < now:
                    self.refs[self.table[a, j]] += 1
            self.lens[b] = self.lens[a]

    def grow(self, slots, add):
        n = len(slots)
        src, dst, granted = [-1] * n, [-1] * n, [0] * n
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        on = {}
        partly = [-1] * n
        for i, (s, a) in enumerate(zip(slots, add)):
            if self.there(s) and a > 0 and self.lens[s] % self.page:
                partly[i] = int(self.table[s, self.up(self.lens[s]) - 1])
                on.setdefault(partly[i], []).append(i)
        begin, given_up = 0, []
        refs = self.refs.copy()
        for i, (s, a) in enumerate(zip(slots, add)):
            if not self.there(s) or a < 0:
                continue
            have = self.up(self.lens[s])
            p = partly[i]
            copy = p >= 0 and refs[p] > 1 and not (len(on[p]) == refs[p] and on[p][-1] == i)
            want = self.up(self.lens[s] + a) - have + copy
            ids = free[begin:begin + want]
            begin += want
            if len(ids) < want or self.lens[s] + a > self.page * self.max_pages:
                continue
            granted[i] = 1
            if copy:
                src[i], dst[i] = p, ids[0]
                given_up.append(p)
                self.table[s, have - 1] = ids[0]
            for j, page in enumerate(ids[int(copy):]):
                self.table[s, have + j] = page
            for page in ids:
                self.refs[page] = 1
            self.lens[s] += a
        for p in given_up:
            self.refs[p] -= 1
        return src, dst, granted

    def compact(self):
        live = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        total = len(live)
        src = [p for p in live if p >= total]
        dst = [p for p in range(total) if self.refs[p] == 0]
        to = np.full(len(self.refs), -1)
        for p in live:
            to[p] = p
        for a, b in zip(src, dst):
            to[a] = b
        refs = np.zeros_like(self.refs)
        for p in live:
            refs[to[p]] = self.refs[p]
        table = np.array([[to[p] if 0 <= p < len(to) else p for p in row] for row in self.table]).reshape(
            self.table.shape)
        return table, refs, to, src, dst
