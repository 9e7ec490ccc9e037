"""dspark_pages_grow where slots that share a partly filled page are refused: a page is kept by one slot only when the
others leave it in the same call, so that no slot writes over another's tokens.  Whole numbers against a restatement,
and the tokens themselves, held in the pages and looked up through the tables."""
import numpy as np
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests import kv4_ref
from tests.test_gpu_kv4_cache import ints
from tests.test_gpu_pages import Both

pytestmark = pytest.mark.gpu


class Pool(kv4_ref.Pool):
    """Growing as include/dspark_kv4.h has it: the last of a page's holders keeps it where all of them are in the list,
    each with tokens that fit its table, and is refused where one of the others is."""

    def fits(self, slot, add):
        return add >= 0 and self.lens[slot] + add <= self.page * self.max_pages

    def grow(self, slots, add):
        n = len(slots)
        src, dst, granted = [-1] * n, [-1] * n, [0] * n
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        refs, partly, leaving = self.refs.copy(), [-1] * n, {}
        for i, (s, a) in enumerate(zip(slots, add)):
            if self.there(s) and a > 0 and self.lens[s] % self.page:
                partly[i] = int(self.table[s, self.up(self.lens[s]) - 1])
                if self.fits(s, a):
                    leaving.setdefault(partly[i], []).append(i)
        begin, given_up = 0, []
        for i, (s, a) in enumerate(zip(slots, add)):
            if not self.there(s) or a < 0:
                continue
            p, have = partly[i], self.up(self.lens[s])
            shared = p >= 0 and refs[p] > 1
            others = leaving.get(p, [])
            keeps = shared and len(others) == refs[p] and others[-1] == i
            copy = shared and not keeps
            want = self.up(self.lens[s] + a) - have + copy
            ids = free[begin:begin + want]
            begin += want
            if len(ids) < want or not self.fits(s, a) or (keeps and not all(granted[j] for j in others[:-1])):
                continue
            granted[i] = 1
            if copy:
                src[i], dst[i] = p, ids[0]
                given_up.append(p)
                self.table[s, have - 1] = ids[0]
            for j, page in enumerate(ids[int(copy):]):
                self.table[s, have + j] = page
            self.refs[ids] = 1
            self.lens[s] += a
        for p in given_up:
            self.refs[p] -= 1
        return src, dst, granted


class Tokens(Both):
    """A pool whose pages hold a number for each token."""

    def __init__(self, num_pages, page, slots, max_pages):
        super().__init__(num_pages, page, slots, max_pages)
        self.ref = Pool(num_pages, page, slots, max_pages)
        self.data = torch.zeros(num_pages, page * 16, dtype=torch.uint8, device="cuda")
        self.held = [[] for _ in range(slots)]
        self.made = 0

    def rows(self):
        return self.data.view(torch.int32).view(self.data.shape[0], self.ref.page, 4)[:, :, 0]

    def step(self, slots, add):
        """Room, copies, and the new tokens of the slots that got room."""
        before = self.ref.lens.copy()
        src, dst, granted = self.grow(slots, add)
        binding.dspark_pages_copy(self.data, ints(src), ints(dst))
        for s, a, ok in zip(slots, add, granted):
            if not ok or a == 0:
                continue
            new = list(range(self.made, self.made + a))
            self.made += a
            at = np.arange(before[s], before[s] + a)
            self.rows()[torch.from_numpy(self.ref.table[s, at // self.ref.page]).cuda(),
                        torch.from_numpy(at % self.ref.page).cuda()] = ints(new)
            self.held[s] += new
        self.look()
        return granted

    def trim(self, slots, new_len):
        super().trim(slots, new_len)
        for s in range(len(self.held)):
            del self.held[s][self.ref.lens[s]:]
        self.look()

    def fork(self, src, dst):
        super().fork(src, dst)
        for a, b in zip(src, dst):
            if self.ref.there(a) and self.ref.there(b) and a != b:
                self.held[b] = list(self.held[a])
        self.look()

    def look(self):
        rows = self.rows().cpu().numpy()
        for s, want in enumerate(self.held):
            at = np.arange(len(want))
            assert rows[self.ref.table[s, at // self.ref.page], at % self.ref.page].tolist() == want, s


@pytest.mark.parametrize("page,max_pages,spare,lens,add,want", [
    (64, 2, 5, (60, 50), (100, 2), [0, 1]),    # the first would exceed its table: the second takes a copy
    (16, 1, 5, (15, 5), (6, 6), [0, 1]),
    (16, 2, 0, (8, 5), (1, 1), [0, 0]),        # no page for the first's copy: the second may not keep the page
    (64, 4, 0, (60, 50), (1, 2), [0, 0]),
    (16, 4, 1, (8, 5), (1, 1), [1, 1]),        # a page for it: the second keeps the shared one
    (16, 4, 1, (8, 5), (9, 1), [0, 0]),        # a copy and a new page are wanted, one is free
    (16, 2, 5, (8, 5), (-1, 1), [0, 1]),
])
def test_a_refused_slot_keeps_its_tokens(page, max_pages, spare, lens, add, want):
    b = Tokens(1 + spare, page, 2, max_pages)
    b.step([0], [lens[0]])
    b.fork([0], [1])
    b.trim([1], [lens[1]])
    assert b.step([0, 1], list(add)) == want


def test_a_slot_alone_gets_its_copy_after_a_refusal():
    b = Tokens(2, 16, 3, 1)
    b.step([0], [12])
    b.fork([0], [1])
    b.trim([1], [9])
    assert b.step([0, 1], [5, 3]) == [0, 0]  # the first does not fit its table, but what it wants counts
    assert b.step([1], [3]) == [1]
    b.trim([1], [0])
    b.fork([0, 0], [1, 2])
    assert b.step([0, 1, 2], [1, 1, 1]) == [1, 0, 0]  # three holders, one free page
    b.trim([0], [0])
    assert b.step([1, 2], [1, 1]) == [1, 1]


@pytest.mark.parametrize("num_pages,page,slots,most,seed", [(12, 16, 6, 3, 0), (14, 64, 12, 2, 1), (10, 32, 8, 2, 2),
                                                           (40, 64, 20, 2, 3)])
def test_the_tokens_of_a_pool_that_is_too_small(num_pages, page, slots, most, seed):
    rng = np.random.default_rng(seed)
    b = Tokens(num_pages, page, slots, most)
    refused = 0
    for _ in range(60):
        chosen = rng.permutation(slots).tolist()
        what = rng.integers(0, 4)
        if what <= 1:
            add = rng.integers(0, page // 2 + 1, slots).tolist()
            granted = b.step(chosen, add)
            refused += granted.count(0)
            for s, a, ok in zip(chosen, add, granted):  # what may be written next is nobody else's
                if ok and a and b.ref.lens[s] % page:
                    assert b.ref.refs[b.ref.table[s, b.ref.up(b.ref.lens[s]) - 1]] == 1
        elif what == 2:
            half = slots // 2
            b.fork(rng.choice(chosen[half:], half).tolist(), chosen[:half])
        else:
            b.trim(chosen, [int(n * rng.random()) for n in b.ref.lens[chosen]])
    assert refused > 0


def test_rows_in_the_cache_of_a_refused_slot():
    """The same through append and read: 64-token pages, the second slot trimmed to 50 of the shared 60 tokens."""
    for max_pages, spare, add in ((2, 3, (100, 2)), (4, 0, (1, 2))):
        b = Tokens(1 + spare, 64, 2, max_pages)
        data = torch.zeros(1 + spare, binding.kv4_page_bytes(64, 2, 64), dtype=torch.uint8, device="cuda")
        cache = binding.Kv4Cache(data, 64, 2, 64)
        x = torch.randn(60, 2, 64, device="cuda").bfloat16()

        def rows(slot, n):
            return binding.Kv4Batch(ints([0, n]), b.lens, b.table, total_rows=n, max_rows=n, slots=ints([slot]))
        b.grow([0], [60])
        binding.dspark_kv4_append(cache, rows(0, 60), x, x)
        b.fork([0], [1])
        Both.trim(b, [1], [50])
        before, after = torch.empty_like(x), torch.empty_like(x)
        binding.dspark_kv4_read(cache, rows(0, 60), before, None)
        src, dst, granted = b.grow([0, 1], list(add))
        binding.dspark_pages_copy(data, ints(src), ints(dst))
        if granted[1]:
            binding.dspark_kv4_append(cache, rows(1, 2), -x[:2], -x[:2])
        binding.dspark_kv4_read(cache, rows(0, 60), after, None)
        assert granted[0] == 0 and torch.equal(before, after)
