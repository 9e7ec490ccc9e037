"""The pages of a cache (dspark_pages_*) against the loops of
tests/kv4_ref.py: whole numbers, equal everywhere."""
import numpy as np
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests import kv4_ref
from tests.test_gpu_kv4_cache import ints

pytestmark = pytest.mark.gpu


class Both:
    """One pool on the GPU and in the restatement."""

    def __init__(self, num_pages, page, slots, max_pages):
        self.ref = kv4_ref.Pool(num_pages, page, slots, max_pages)
        self.refs, self.table, self.lens = ints(self.ref.refs), ints(self.ref.table), ints(self.ref.lens)
        self.pool = binding.PagePool(self.refs, self.table, self.lens, page)

    def same(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.lens.cpu().numpy(), self.ref.lens)
        assert np.array_equal(self.refs.cpu().numpy(), self.ref.refs)
        assert np.array_equal(self.table.cpu().numpy(), self.ref.table)

    def grow(self, slots, add):
        out = [ints([7] * len(slots)) for _ in range(3)]
        binding.dspark_pages_grow(self.pool, ints(slots), ints(add), *out)
        want = self.ref.grow(slots, add)
        self.same()
        got = [o.cpu().tolist() for o in out]
        assert got == [list(w) for w in want]
        return got

    def trim(self, slots, new_len):
        binding.dspark_pages_trim(self.pool, ints(slots), ints(new_len))
        self.ref.trim(slots, new_len)
        self.same()

    def fork(self, src, dst):
        binding.dspark_pages_fork(self.pool, ints(src), ints(dst))
        self.ref.fork(src, dst)
        self.same()

    def compact(self, in_place):
        n = self.refs.numel()
        table, refs = (self.table, self.refs) if in_place else (torch.empty_like(self.table), ints([9] * n))
        to, src, dst, count = ints([9] * n), ints([9] * n), ints([9] * n), ints([9])
        want_table, want_refs, want_to, want_src, want_dst = self.ref.compact()
        binding.dspark_pages_compact(self.pool, table, refs, to, src, dst, count)
        torch.cuda.synchronize()
        m = len(want_src)
        assert count.item() == m == len(want_dst)
        assert src.cpu().tolist() == want_src + [-1] * (n - m)
        assert dst.cpu().tolist() == want_dst + [-1] * (n - m)
        assert np.array_equal(to.cpu().numpy(), want_to)
        assert np.array_equal(table.cpu().numpy(), want_table) and np.array_equal(refs.cpu().numpy(), want_refs)
        if in_place:
            self.ref.table, self.ref.refs = want_table, want_refs
        self.same()


@pytest.mark.parametrize("num_pages,page,slots,seed", [(64, 16, 6, 0), (1000, 16, 40, 1), (5003, 4, 70, 2),
                                                       (300, 1, 9, 3), (20000, 64, 300, 4)])
def test_a_random_life_of_a_pool(num_pages, page, slots, seed):
    """Growing (with too little room at times), forking, trimming and compacting in random order."""
    rng = np.random.default_rng(seed)
    most = min(64, max(4, 2 * num_pages // slots))
    b = Both(num_pages, page, slots, most)
    for step in range(40):
        n = int(rng.integers(1, slots + 1))
        chosen = rng.permutation(slots + 2)[:n] - 1  # one below and one behind the slots among them
        what = rng.integers(0, 5)
        if what <= 1:
            b.grow(chosen.tolist(), rng.integers(-1, 3 * page + 2, n).tolist())
        elif what == 2:
            half = n // 2
            b.fork(rng.choice(chosen[half:], half).tolist() if half else [], chosen[:half].tolist())
        elif what == 3:
            b.trim(chosen.tolist(), rng.integers(-1, most * page // 2, n).tolist())
        else:
            b.compact(bool(rng.integers(0, 2)))


def test_branches_copy_a_shared_last_page_once_each():
    b = Both(50, 16, 8, 10)
    b.grow([0], [40])
    b.fork([0, 0, 0], [3, 4, 5])
    src, dst, granted = b.grow([3, 4, 5, 0], [6, 6, 6, 6])
    assert src == [2, 2, 2, -1] and dst == [3, 4, 5, -1] and granted == [1] * 4  # the last holder keeps the page
    b.trim([3, 4, 5, 0], [0, 0, 0, 43])
    b.fork([0, 0], [3, 4])
    src, dst, _ = b.grow([3, 4], [1, 1])  # slot 0 holds the page too and is not in the list
    assert src == [2, 2]
    b.trim([3, 4], [0, 0])
    src, dst, _ = b.grow([0], [1])
    assert src == [-1] and dst == [-1]


def test_a_full_page_is_shared_and_never_copied():
    b = Both(50, 16, 4, 10)
    b.grow([0], [32])
    b.fork([0], [1])
    src, _, _ = b.grow([0, 1], [1, 1])
    assert src == [-1, -1]


def test_grants_go_in_order_and_stop_where_the_pages_do():
    b = Both(10, 16, 8, 6)
    assert b.grow([0, 1, 2, 3], [64, 64, 64, 0])[2] == [1, 1, 0, 1]
    assert b.grow([4, 5, 6], [16, 32, 16])[2] == [1, 0, 0]  # what a slot wants counts even if it is not granted
    assert b.grow([0, 6], [64, 16])[2] == [0, 0]            # slot 0 would exceed its 6 pages
    b2 = Both(3, 16, 2, 1 << 12)
    assert b2.grow([0, 1], [2 ** 16 - 1, 5])[2] == [0, 0]
    assert b2.grow([0], [2 ** 31 - 1])[2] == [0]


def test_many_slots_and_a_large_pool():
    n = binding.PAGES_MAX_SLOTS
    b = Both(100001, 16, n, 8)
    rng = np.random.default_rng(1)
    order = rng.permutation(n)
    b.grow(order.tolist(), rng.integers(0, 60, n).tolist())
    half = n // 2
    b.fork(order[:half].tolist(), order[half:].tolist())
    b.grow(order[::-1].tolist(), rng.integers(0, 40, n).tolist())
    b.compact(True)


def test_unaligned_arrays():
    """Reference counts that do not start on 16 bytes."""
    b = Both(700, 16, 9, 30)
    held = torch.zeros(701, dtype=torch.int32, device="cuda")
    b.refs = held[1:]
    b.pool = binding.PagePool(b.refs, b.table, b.lens, 16)
    b.grow(list(range(9)), [100] * 9)
    b.trim([1, 3, 5], [0, 0, 0])
    b.compact(False)
    b.compact(True)
    assert held[0] == 0


@pytest.mark.parametrize("layers,pages,size,n", [(1, 20, 16, 3), (3, 40, 2304, 20), (2, 9, 73728, 4), (1, 300, 9216, 150)])
def test_copying_pages(layers, pages, size, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    wide = torch.randint(0, 256, (layers, pages, size + 32), dtype=torch.uint8, device="cuda", generator=g)
    data = wide[:, :, :size]
    ids = torch.randperm(pages, generator=torch.Generator().manual_seed(n))[:2 * n].tolist()
    src, dst = ids[:n], ids[n:]
    if n > 2:
        src[1], dst[2] = -1, pages + 7  # skipped
    want = wide.clone()
    for a, b in zip(src, dst):
        if 0 <= a < pages and 0 <= b < pages:
            want[:, b, :size] = want[:, a, :size]
    first = wide.clone()
    binding.dspark_pages_copy(data, ints(src), ints(dst))
    assert torch.equal(wide, want)
    wide.copy_(first)
    binding.dspark_pages_copy(data, ints(src), ints(dst), count=ints([1]))
    want = first.clone()
    want[:, dst[0], :size] = first[:, src[0], :size]
    assert torch.equal(wide, want)
    wide.copy_(first)
    for c in (0, -3):
        binding.dspark_pages_copy(data, ints(src), ints(dst), count=ints([c]))
        assert torch.equal(wide, first)


def test_copying_behind_4_gib():
    size = 1 << 20
    data = torch.zeros(4100, size, dtype=torch.uint8, device="cuda")
    data[4098] = 7
    binding.dspark_pages_copy(data, ints([4098]), ints([4099]))
    assert torch.all(data[4099] == 7) and not data[:4098].any()


def test_a_captured_round():
    """Trim, fork, grow and copy in one CUDA graph, replayed."""
    b = Both(200, 16, 8, 20)
    b.grow([0, 1], [100, 33])
    data = torch.randint(0, 256, (200, 2304), dtype=torch.uint8, device="cuda")
    every, base, add = ints([2, 3, 0, 1]), ints([0, 0, 100, 33]), ints([6] * 4)
    src, dst = ints([0, 1]), ints([2, 3])
    cs, cd, ok = ints([0] * 4), ints([0] * 4), ints([0] * 4)
    graph = torch.cuda.CUDAGraph()

    def one():
        binding.dspark_pages_trim(b.pool, every, base)
        binding.dspark_pages_fork(b.pool, src, dst)
        binding.dspark_pages_grow(b.pool, every, add, cs, cd, ok)
        binding.dspark_pages_copy(data, cs, cd)
    one()
    torch.cuda.synchronize()
    state = [t.clone() for t in (b.refs, b.table, b.lens, cs, cd, ok)]
    with torch.cuda.graph(graph):
        one()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(state, (b.refs, b.table, b.lens, cs, cd, ok)))
    assert ok.tolist() == [1] * 4 and b.lens[:4].tolist() == [106, 39, 106, 39]
