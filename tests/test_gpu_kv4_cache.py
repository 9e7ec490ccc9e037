"""Storing rows in the paged 4-bit cache and reading them back, against the
64-bit restatement of tests/kv4_ref.py.

Codes and scales are decided by comparing correctly rounded FP32 quotients with
the formats' grids.  With power-of-two head scales those decisions equal the
exact ones (x has at most 11 significant bits, a scale 4: a quotient that is not
on a tie is further from it than FP32's rounding), so every byte of the cache
must be equal.  With other head scales y = x / g has 24 bits and a quotient may
round onto a tie: a byte may then differ, where the exact quotient lies within
2^-22 of one.  Values read are one FP32 product, rounded once more."""
import numpy as np
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests import kv4_ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, rows, lens, page, heads, dim, *, dtype="bf16", gk=None, gv=None, seed=0, slots=None, spread=1.0):
        rng = np.random.default_rng(seed)
        self.rows, self.lens, self.dim, self.heads, self.page = rows, lens, dim, heads, page
        self.start = np.concatenate([[0], np.cumsum(rows)]).astype(int)
        self.total = int(self.start[-1])
        self.slots = list(range(len(rows))) if slots is None else slots
        slot_lens = np.zeros(max(self.slots) + 2, int)
        for s, n in zip(self.slots, lens):
            slot_lens[s] = n
        need = [-(-n // page) for n in slot_lens]
        num_pages = sum(need) + 3
        ids = rng.permutation(num_pages)
        self.table = np.full((len(slot_lens), max(max(need), 1) + 1), -1)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = ids[at:at + n]
            at += n
        self.slot_lens = slot_lens
        self.ref = kv4_ref.Cache(num_pages, page, heads, dim, gk, gv, rng)
        f32 = lambda g: None if g is None else torch.tensor(g, dtype=torch.float32, device="cuda")  # noqa: E731
        self.data = torch.from_numpy(self.ref.data.copy()).cuda()
        self.cache = binding.Kv4Cache(self.data, page, heads, dim, k_scale=f32(gk), v_scale=f32(gv))
        self.batch = binding.Kv4Batch(ints(self.start), ints(slot_lens), ints(self.table), total_rows=self.total,
                                      max_rows=max(rows), slots=None if slots is None else ints(slots))
        x = rng.standard_normal((2, self.total, heads, dim)) * np.exp(spread * rng.standard_normal((1, 1, heads, dim)))
        self.k, self.v = (torch.from_numpy(t).to(TYPES[dtype]).cuda() for t in x)

    def where(self):
        """(row, page, row in the page) of the rows that have a place."""
        for i, s in enumerate(self.slots):
            for j in range(self.rows[i]):
                pos = self.slot_lens[s] - self.rows[i] + j
                if pos >= 0:
                    p = self.table[s, pos // self.page]
                    if 0 <= p < self.ref.num_pages:
                        yield self.start[i] + j, p, pos % self.page

    def store(self):
        k, v = self.k.double().cpu().numpy(), self.v.double().cpu().numpy()
        for row, p, r in self.where():
            self.ref.store(p, r, k[row], v[row])


CASES = [
    dict(rows=[1], lens=[1], page=16, heads=1, dim=64),
    dict(rows=[6, 6, 6], lens=[100, 6, 71], page=64, heads=8, dim=128),
    dict(rows=[0, 1, 0, 33, 2], lens=[5, 17, 0, 33, 1], page=16, heads=5, dim=64, dtype="f16"),
    dict(rows=[5, 7], lens=[3, 300], page=256, heads=2, dim=128, gk=[0.25, 4.0], gv=[1.0, 2.0 ** -7]),
    dict(rows=[129, 1], lens=[200, 257], page=32, heads=3, dim=128, slots=[4, 1], dtype="f16"),
    dict(rows=[40], lens=[40], page=128, heads=1, dim=64, spread=6.0),
]


@pytest.mark.parametrize("kw", CASES)
def test_append_writes_the_exact_bytes_and_no_others(kw):
    c = Case(**kw)
    c.store()
    binding.dspark_kv4_append(c.cache, c.batch, c.k, c.v)
    torch.cuda.synchronize()
    got = c.data.cpu().numpy()
    # a code's sign where the magnitude is 0 is free
    same = got == c.ref.data
    if not same.all():
        for p, at in np.argwhere(~same):
            r = at % c.ref.record
            assert r < c.page * c.dim, "a scale differs"
            a, b = int(got[p, at]), int(c.ref.data[p, at])
            for sh in (0, 4):
                x, y = a >> sh & 15, b >> sh & 15
                assert x == y or (x & 7) == (y & 7) == 0, (p, at, a, b)


@pytest.mark.parametrize("kw", CASES)
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_read_gives_the_values(kw, out):
    c = Case(**kw)
    dtype = dict(TYPES, f32=torch.float32)[out]
    k = torch.full((c.total, c.heads, c.dim), -77.0, dtype=dtype, device="cuda")
    v = torch.full_like(k, -77.0)
    binding.dspark_kv4_read(c.cache, c.batch, k, v)
    want = np.zeros((2, c.total, c.heads, c.dim))
    for row, p, r in c.where():
        for h in range(c.heads):
            want[0, row, h], want[1, row, h] = c.ref.load(p, r, h)
    # the pool's random bytes: code * scale is exact, the product with a power of two too
    for got, w in ((k, want[0]), (v, want[1])):
        assert torch.equal(got.cpu(), torch.from_numpy(w).float().to(dtype))


def test_head_scales_off_the_grid():
    """Any finite head scale: scales and codes equal but for quotients that FP32 rounds onto a tie."""
    rng = np.random.default_rng(5)
    gk, gv = (np.exp(rng.standard_normal(4)).astype(np.float32).tolist() for _ in range(2))
    c = Case([200], [200], 64, 4, 128, gk=gk, gv=gv, seed=6)
    binding.dspark_kv4_append(c.cache, c.batch, c.k, c.v)
    k32 = torch.empty(c.total, c.heads, c.dim, device="cuda")
    v32 = torch.empty_like(k32)
    binding.dspark_kv4_read(c.cache, c.batch, k32, v32)
    for x, got, g in ((c.k, k32, gk), (c.v, v32, gv)):
        x, got, g = x.double().cpu().numpy(), got.double().cpu().numpy(), np.asarray(g)[None, :, None]
        code, scale = kv4_ref.quantise(x, g)
        want = kv4_ref.values(code, scale, g)
        off = np.abs(got - want) > 2.0 ** -23 * np.abs(want)
        assert off.mean() < 1e-4
        s = np.repeat(kv4_ref.POSITIVE[scale], 16, -1)
        ratio = np.abs(x / g / s)[off]
        ties = (kv4_ref.E2M1[1:] + kv4_ref.E2M1[:-1]) / 2
        near = np.abs(ratio[:, None] / ties[None] - 1).min(-1)
        assert np.all(near < 2.0 ** -22), near.max()


def test_infinities_nan_zeros_and_the_smallest():
    c = Case([6], [6], 16, 1, 64)
    x = torch.zeros(6, 1, 64)
    x[0, 0, 3] = float("nan")
    x[0, 0, 4] = 3.0
    x[1, 0, 0], x[1, 0, 1], x[1, 0, 2] = float("inf"), -float("inf"), 1000.0
    x[2, 0, :16] = float("nan")
    x[3] = 2.0 ** -14
    x[4, 0, 20] = 3.0e38
    x[5] = -0.0
    c.k = c.v = x.to(torch.bfloat16).cuda()
    c.store()
    binding.dspark_kv4_append(c.cache, c.batch, c.k, c.v)
    k = torch.empty(6, 1, 64, device="cuda")
    binding.dspark_kv4_read(c.cache, c.batch, k, None)
    k = k.cpu()
    assert torch.isfinite(k).all()
    assert k[0, 0, 3] == 0 and k[0, 0, 4] == 3.0
    assert k[1, 0, 0] == 2688.0 and k[1, 0, 1] == -2688.0 and k[1, 0, 2] == 896.0  # 1000 / 448 = 2.23
    assert torch.all(k[2] == 0) and torch.all(k[3] == 0) and torch.all(k[5] == 0)
    assert k[4, 0, 20] == 2688.0


def test_strided_and_unaligned_rows():
    """Rows inside a wider projection (16-byte aligned or not) give the bytes that contiguous rows give."""
    base = Case([6, 3], [40, 3], 16, 2, 128)
    binding.dspark_kv4_append(base.cache, base.batch, base.k, base.v)
    for offset in (0, 8, 1):
        c = Case([6, 3], [40, 3], 16, 2, 128)
        wide = torch.zeros(c.total, 3 * 2 * 128 + 16 + offset, dtype=torch.bfloat16, device="cuda")
        flat = wide[:, offset:offset + 3 * 256].unflatten(1, (2, 3, 128))
        k, v = flat[:, :, 1], flat[:, :, 2]
        k.copy_(base.k)
        v.copy_(base.v)
        binding.dspark_kv4_append(c.cache, c.batch, k, v)
        assert torch.equal(c.data, base.data)
        ko, vo = torch.zeros_like(wide), torch.zeros(c.total, 2, 128, dtype=torch.bfloat16, device="cuda")
        ko_v = ko[:, offset:offset + 3 * 256].unflatten(1, (2, 3, 128))[:, :, 1]
        want_k, want_v = torch.empty_like(base.k), torch.empty_like(base.v)
        binding.dspark_kv4_read(c.cache, c.batch, ko_v, vo)
        binding.dspark_kv4_read(base.cache, base.batch, want_k, want_v)
        assert torch.equal(ko_v, want_k) and torch.equal(vo, want_v)
        ko_v.zero_()
        assert not ko.any()  # nothing beside the rows was written


def test_rows_without_a_place():
    """Rows at negative positions, of slots that are not there, on pages that are not there: not stored, read as 0;
    rows of no request: not touched."""
    c = Case([4, 2, 3], [2, 40, 33], 16, 1, 64)
    c.table[1, 2] = -1          # the page of request 1's rows
    c.table[2, 2] = 10 ** 6     # page id out of range for request 2's last row
    start = ints([1, 5, 7, 10])  # row 0 and rows from 10 on belong to nobody
    c.batch = binding.Kv4Batch(start, ints(c.slot_lens), ints(c.table), total_rows=12, max_rows=4,
                               slots=ints([0, 1, 2]))
    k = torch.randn(12, 1, 64, device="cuda").to(torch.bfloat16)
    before = c.data.clone()
    binding.dspark_kv4_append(c.cache, c.batch, k, k)
    changed = (c.data != before).any(1).nonzero().flatten().tolist()
    assert set(changed) <= {c.table[0, 0], c.table[2, 1]}
    out = torch.full((12, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    binding.dspark_kv4_read(c.cache, c.batch, out, None)
    there = {3, 4, 7, 8}  # request 0: positions -2 .. 1; request 2: 30, 31 on a page, 32 on none
    for row in range(12):
        if row in (0, 10, 11):
            assert torch.all(out[row] == 5.0)
        elif row not in there:
            assert torch.all(out[row] == 0.0), row
    bad = binding.Kv4Batch(ints([0, 4]), ints(c.slot_lens), ints(c.table), total_rows=4, max_rows=4, slots=ints([99]))
    before = c.data.clone()
    binding.dspark_kv4_append(c.cache, bad, k, k)
    assert torch.equal(before, c.data)


def test_pages_of_a_wider_pool_and_far_offsets():
    """A page stride larger than the page (layers side by side), and a pool of more than 2^32 bytes."""
    page, heads, dim = 64, 2, 128
    size = binding.kv4_page_bytes(page, heads, dim)
    pages = (1 << 32) // (3 * size) + 10
    pool = torch.zeros(pages, 3 * size, dtype=torch.uint8, device="cuda")
    layer = pool[:, size:2 * size]
    cache = binding.Kv4Cache(layer, page, heads, dim)
    batch = binding.Kv4Batch(ints([0, 64]), ints([64]), ints([[pages - 1]]), total_rows=64, max_rows=64)
    x = torch.randn(64, heads, dim, device="cuda").to(torch.bfloat16)
    binding.dspark_kv4_append(cache, batch, x, -x)
    k, v = torch.empty_like(x), torch.empty_like(x)
    binding.dspark_kv4_read(cache, batch, k, v)
    assert torch.equal(k, -v) and (k - x).abs().max() < 0.6
    assert layer[pages - 1].any() and not pool[:pages - 1].any()
    assert not pool[pages - 1, :size].any() and not pool[pages - 1, 2 * size:].any()
