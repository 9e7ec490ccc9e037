"""What the eight bits of bounds and of queries can cost a selection (the kernels' lists are tests/select_ref.py's, page
for page): no page that is left out has a score by unrounded bounds that is above that of a page kept by more than the two
pages' roundings.  No GPU needed.

With x the keys of a page, m the largest |x|, a and b the sums of a group's negative and positive parts, t the largest of
those: lo = (m / 127) (lo8 + d), |d| <= 1 / 2, and a = (t / 127) (a8 + e), |e| <= 1 / 2 (each by 2^-15 more, for the FP32
product and quotient before the rounding).  So |a lo - (m t / 127^2) a8 lo8| <= |a| m / 254 + (|lo| + m / 254) t / 254, the
same for b hi, and a score is their sum over the dimensions, rounded once to FP32."""
import numpy as np
import pytest

from tests import kv4_ref, select_ref

MORE = 1 + 2.0 ** -15


@pytest.mark.parametrize("dim,group,page", [(64, 1, 16), (128, 8, 64), (64, 5, 32)])
@pytest.mark.parametrize("kind", ["alike", "two large", "two large, queries small there"])
def test_pages_left_out_are_within_the_roundings(dim, group, page, kind):
    rng = np.random.default_rng(dim + group)
    pages, top, first, last = 150, 20, 1, 2
    keys, queries = np.ones(dim), np.ones(dim)
    if kind != "alike":
        keys[[3, dim - 5]] = 10, 20
    if kind == "two large, queries small there":
        queries = 1 / keys
    cache = kv4_ref.Cache(pages, page, 1, dim, rng=rng)
    common = rng.standard_normal((pages, 1, dim))  # tokens of a page resemble one another
    x = (rng.standard_normal((pages, page, dim)) + 0.7 * common) * keys
    for p in range(pages):
        for r in range(page):
            cache.store(p, r, x[p, r][None], x[p, r][None])
    bounds = np.stack([select_ref.record_of(*select_ref.bounds_of(cache, p, 0, page)) for p in range(pages)])
    q = (rng.standard_normal((group, dim)) * queries).astype(np.float32)
    kept = select_ref.select(bounds, pages, page, np.arange(pages), pages * page - 1, q, False, dim, top, first, last)
    assert len(kept) == top
    held = np.stack([np.stack([cache.load(p, r, 0)[0] for r in range(page)]) for p in range(pages)])
    lo, hi = held.min(1), held.max(1)
    a, b = np.minimum(q, 0).sum(0, dtype=np.float64), np.maximum(q, 0).sum(0, dtype=np.float64)
    m, t = np.maximum(np.abs(lo), np.abs(hi)).max(1), max(np.abs(a).max(), b.max())
    exact = lo @ a + hi @ b
    off = MORE * (m / 254 * (np.abs(a) + b).sum() + t / 254 * (np.abs(lo) + np.abs(hi) + 2 * MORE * m[:, None] / 254).sum(1))
    off += 2.0 ** -23 * (np.abs(exact) + off) + group * 2.0 ** -23 * ((np.abs(lo) @ -a) + np.abs(hi) @ b)  # FP32's sums, too
    free = [p for p in kept if first <= p < pages - last]
    left = [p for p in range(pages) if p not in kept]
    for p in free:
        assert np.all(exact[left] <= exact[p] + off[left] + off[p])
