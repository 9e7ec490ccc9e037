"""Plain restatement of page bounds, selection and attention over a selection (include/dspark_kv4.h).  Test
infrastructure only."""
import numpy as np

from tests import kv4_ref

F = np.float32


def bounds_of(cache, page, head, held):
    """lo, hi (int8) and m of the page's first `held` keys."""
    codes, scales = cache.sections(page, head)
    b = codes[0][:held]
    code = np.stack([b & 15, b >> 4], -1).reshape(held, -1)
    x = kv4_ref.values(code, scales[0][:held], 1.0)
    lo, hi = x.min(0), x.max(0)
    m = max(np.abs(lo).max(), np.abs(hi).max())
    if m == 0:
        return np.zeros(len(lo), np.int8), np.zeros(len(lo), np.int8), F(0)
    part = [np.rint((F(127) * y.astype(F)) / F(m)).astype(np.int8) for y in (lo, hi)]
    return part[0], part[1], F(m)


def record_of(lo, hi, m):
    return np.concatenate([lo.view(np.uint8), hi.view(np.uint8), np.array([m], F).view(np.uint8), np.zeros(12, np.uint8)])


def parts_of(q, negative):
    """q FP32 [group, dim] -> a, b int64 [dim]."""
    q = np.where(np.isnan(q), F(0), np.clip(q, F(-2.0 ** 100), F(2.0 ** 100))).astype(F)
    if negative:
        q = -q
    a, b = np.zeros(q.shape[1], F), np.zeros(q.shape[1], F)
    for row in q:
        a, b = a + np.minimum(row, F(0)), b + np.maximum(row, F(0))
    top = max(np.abs(a).max(), b.max())
    if top == 0:
        return np.zeros(q.shape[1], np.int64), np.zeros(q.shape[1], np.int64)
    return tuple(np.rint((F(127) * x) / top).astype(np.int64) for x in (a, b))


def select(bounds, num_pages, page, table, pos, q, negative, dim, top, first, last):
    """The page ids of one row and head.  bounds: this head's records, uint8 [num_pages, 2 dim + 16]."""
    n = pos // page + 1
    if n <= top:
        return [int(p) for p in table[:n]]
    a, b = parts_of(q, negative)
    score = np.full(n, -np.inf)
    for p in range(n):
        if 0 <= table[p] < num_pages:
            rec = bounds[table[p]]
            lo, hi = rec[:dim].view(np.int8).astype(np.int64), rec[dim:2 * dim].view(np.int8).astype(np.int64)
            score[p] = rec[2 * dim:2 * dim + 4].copy().view(F)[0] * F(int(a @ lo + b @ hi))
    score[:first] = np.inf
    score[n - last:] = np.inf
    order = np.argsort(-score, kind="stable")[:top]
    return [int(table[p]) for p in np.sort(order)]


class OneHead:
    """A head of a kv4_ref.Cache as a cache of one head."""

    def __init__(self, cache, head):
        self.cache, self.head, self.page, self.heads, self.dim = cache, head, cache.page, 1, cache.dim

    def tokens(self, pages, length, head):
        return self.cache.tokens(pages, length, self.head)


def attention(cache, pages, lens, q, group, scale):
    """kv4_ref.attention over a selection: pages [rows, heads, top], lens [rows]."""
    rows, heads, _ = pages.shape
    out = [kv4_ref.attention(OneHead(cache, h), np.arange(rows + 1), np.arange(rows), np.maximum(lens, 0), pages[:, h],
                             q[:, h * group:(h + 1) * group], group, scale, 0) for h in range(heads)]
    return tuple(np.concatenate([o[i] for o in out], 1) for i in range(3))
