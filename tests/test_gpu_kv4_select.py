"""Bounds of pages and the pages that rows select, against tests/select_ref.py: whole numbers, all equal; attention
over a selection against 64 bits within the bound of kv4_ref.attention."""
import numpy as np
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests import select_ref
from tests.test_gpu_kv4_attention import Case as Attention
from tests.test_gpu_kv4_cache import ints

pytestmark = pytest.mark.gpu


class Case(Attention):
    def __init__(self, rows, lens, page, heads, group, dim, *, top, first=1, last=1, **kw):
        super().__init__(rows, lens, page, heads, group, dim, **kw)
        self.page, self.top, self.first, self.last = page, top, first, last
        size = binding.kv4_bounds_bytes(heads, dim)
        rng = np.random.default_rng(3)
        self.ref_bounds = rng.integers(0, 256, (self.ref.num_pages, size), dtype=np.uint8)  # NaN and all
        self.bounds = torch.from_numpy(self.ref_bounds.copy()).cuda()
        self.pages = torch.full((self.total, heads, top), -77, dtype=torch.int32, device="cuda")
        self.kept = torch.full((self.total,), -77, dtype=torch.int32, device="cuda")
        self.selection = binding.Kv4Selection(self.pages, self.kept)

    def scratch(self, n):
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def bound_all(self):
        """Bounds of every page of the tables, a request at a time, as prompts would leave them."""
        for s in range(len(self.lens)):
            n = int(self.lens[s])
            batch = binding.Kv4Batch(ints([0, n]), ints(self.lens), ints(self.table), total_rows=n, max_rows=n,
                                     slots=ints([s]))
            binding.dspark_kv4_bound_pages(self.cache, batch, self.bounds)
            for p in range(-(-n // self.page)):
                self.put(s, p)

    def put(self, slot, p):
        page = self.table[slot, p]
        if not 0 <= page < self.ref.num_pages:
            return
        held = min(self.page, int(self.lens[slot]) - p * self.page)
        r = self.ref_bounds[page].reshape(self.heads, -1)
        for h in range(self.heads):
            r[h] = select_ref.record_of(*select_ref.bounds_of(self.ref, page, h, held))

    def select(self, q=None):
        q = self.q if q is None else q
        size = binding.dspark_kv4_select_workspace_bytes(self.cache, self.batch, self.selection)
        binding.dspark_kv4_select(self.cache, self.batch, self.bounds, q, self.selection, self.scratch(size),
                                  first=self.first, last=self.last)
        torch.cuda.synchronize()
        return self.pages.cpu().numpy(), self.kept.cpu().numpy()

    def wanted(self):
        pages = np.full((self.total, self.heads, self.top), -1)
        kept = np.full(self.total, -1)
        q = self.q.float().cpu().numpy()
        for i, s in enumerate(self.slots):
            n = int(self.lens[s]) if 0 <= s < len(self.lens) else 0
            for j in range(self.rows[i]):
                row, pos = self.start[i] + j, n - self.rows[i] + j
                kept[row] = 0
                if pos < 0:
                    continue
                for h in range(self.heads):
                    b = self.ref_bounds.reshape(self.ref.num_pages, self.heads, -1)[:, h]
                    g = self.ref.g[0][h] < 0
                    ids = select_ref.select(b, self.ref.num_pages, self.page, self.table[s], pos,
                                            q[row, h * self.group:(h + 1) * self.group], g, self.dim, self.top,
                                            self.first, self.last)
                    pages[row, h, :len(ids)] = ids
                kept[row] = (min(pos // self.page + 1, self.top) - 1) * self.page + pos % self.page + 1
        return pages, kept

    def attend(self, lse=True):
        out = torch.full_like(self.q, -55.0)
        lse = torch.full((self.total, self.heads * self.group), -55.0, device="cuda") if lse else None
        size = binding.dspark_kv4_attention_selected_workspace_bytes(self.cache, self.selection, self.heads * self.group)
        binding.dspark_kv4_attention_selected(self.cache, self.selection, self.q, out, self.scale, self.scratch(size),
                                              lse=lse)
        torch.cuda.synchronize()
        return out, lse

    def check_attention(self):
        pages, kept = self.pages.cpu().numpy(), self.kept.cpu().numpy()
        out, lse = self.attend()
        want, want_lse, tol = select_ref.attention(self.ref, pages, kept, self.q.double().cpu().numpy(), self.group,
                                                   self.scale)
        got = out.double().cpu().numpy()
        there = kept >= 0
        unit = 2.0 ** -9 if self.dtype == "bf16" else 2.0 ** -12
        room = 2 * (tol + unit * np.abs(want)) + 2.0 ** -24
        assert np.all((np.abs(got - want) <= room)[there])
        assert np.all(got[~there] == -55.0)
        got = lse.double().cpu().numpy()
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got[there]), empty[there])
        d = 2.0 ** -20 * (1 + np.abs(want_lse[~empty])) + tol[~empty].max(initial=0)  # as for whole caches
        assert np.all(np.abs(got[~empty] - want_lse[~empty]) <= d)


CASES = [
    dict(rows=[1], lens=[1], page=16, heads=1, group=1, dim=64, top=1, first=0),
    dict(rows=[1], lens=[200], page=16, heads=1, group=8, dim=128, top=5, first=1, last=2),
    dict(rows=[1, 1, 1], lens=[64, 129, 640], page=64, heads=2, group=4, dim=128, top=2),
    dict(rows=[6, 6], lens=[300, 6], page=16, heads=2, group=8, dim=128, top=7, first=2, last=3),
    dict(rows=[0, 3, 1, 17], lens=[50, 2, 400, 333], page=16, heads=5, group=5, dim=64, top=4, dtype="f16", slots=[3, 1, 0, 5]),
    dict(rows=[6], lens=[500], page=32, heads=2, group=3, dim=64, top=9, first=0, last=1, gk=[-0.3, 2.0], gv=[1.0, -0.5]),
    dict(rows=[40], lens=[700], page=16, heads=1, group=2, dim=128, top=3),
    dict(rows=[2], lens=[2000], page=256, heads=2, group=16, dim=64, top=6, last=2, dtype="f16"),
    dict(rows=[3], lens=[900], page=128, heads=1, group=20, dim=128, top=4),
    dict(rows=[2, 2], lens=[100, 0], page=16, heads=2, group=2, dim=64, top=100),
    dict(rows=[2, 1], lens=[16 * 639 + 3, 16 * 512], page=16, heads=1, group=2, dim=64, top=50),
    dict(rows=[2], lens=[16 * 1500 + 3], page=16, heads=1, group=2, dim=128, top=70, last=3),
    dict(rows=[6, 6, 0], lens=[16 * 620, 9000, 0], page=16, heads=3, group=1, dim=64, top=20, dtype="f16"),
    dict(rows=[1, 2], lens=[16 * 2048, 3], page=16, heads=1, group=1, dim=64, top=2047, first=2000, last=40),
]


# tables much wider than the requests are long take the three launches for short requests, too
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kw", CASES)
def test_bounds_selection_and_attention(kw, wide):
    c = Case(wide=wide, **kw)
    c.bound_all()
    torch.cuda.synchronize()
    assert np.array_equal(c.bounds.cpu().numpy(), c.ref_bounds)
    got, want = c.select(), c.wanted()
    assert np.array_equal(got[1], want[1])
    assert np.array_equal(got[0], want[0])
    c.check_attention()


def test_bounds_of_the_steps_pages_only():
    c = Case(rows=[3, 1, 0], lens=[66, 64, 20], page=16, heads=2, group=2, dim=64, top=3)
    binding.dspark_kv4_bound_pages(c.cache, c.batch, c.bounds)
    for s, p in ((0, 3), (0, 4), (1, 3)):  # rows 63, 64, 65 and 63
        c.put(s, p)
    assert np.array_equal(c.bounds.cpu().numpy(), c.ref_bounds)


def test_bounds_of_pages_of_zeros_and_of_any_bytes():
    c = Case(rows=[48], lens=[48], page=16, heads=2, group=2, dim=64, top=3, normal=False)
    data = c.ref.data
    data[c.table[0, 1]] = 0
    c.data.copy_(torch.from_numpy(data))
    c.bound_all()
    assert np.array_equal(c.bounds.cpu().numpy(), c.ref_bounds)


@pytest.mark.parametrize("many", [2100, 9000, 13000])
def test_many_pages_and_ties(many):
    """More pages than registers hold keys for, and more than shared memory does; equal scores go to the lower pages."""
    c = Case(rows=[2], lens=[16 * many + 5], page=16, heads=1, group=1, dim=64, top=300, first=3, last=2, normal=False)
    c.ref_bounds[:] = 0
    rng = np.random.default_rng(1)
    kinds = [select_ref.record_of(*(rng.integers(-127, 128, 64).astype(np.int8) for _ in range(2)), np.float32(m))
             for m in (0.5, 1.0, 3.0)]
    c.ref_bounds[:] = np.stack(kinds)[rng.integers(0, 3, len(c.ref_bounds))]
    c.bounds.copy_(torch.from_numpy(c.ref_bounds))
    got, want = c.select(), c.wanted()
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("what", ["zero", "nan", "inf", "huge", "tiny"])
def test_queries_of_zeros_nan_and_infinities(what, wide):
    c = Case(rows=[2], lens=[400], page=16, heads=2, group=2, dim=64, top=5, wide=wide)
    c.bound_all()
    if what == "zero":
        c.q.zero_()
    elif what == "nan":
        c.q[:, :, ::3] = float("nan")
    elif what == "inf":
        c.q[0, :, 5], c.q[1, 1, 7] = float("inf"), float("-inf")
    elif what == "huge":
        c.q.fill_(torch.finfo(torch.bfloat16).max)
    else:
        c.q.mul_(2.0 ** -130)
    got, want = c.select(), c.wanted()
    assert np.array_equal(got[0], want[0])


@pytest.mark.parametrize("wide", [False, True])
def test_pages_that_are_not_there_come_last(wide):
    def holes(table, num_pages):
        table[0, 3:6] = [-1, num_pages, 2 ** 30]
        table[0, 24] = -5
    c = Case(rows=[3], lens=[400], page=16, heads=2, group=2, dim=64, top=23, table=holes, wide=wide)
    c.bound_all()
    got, want = c.select(), c.wanted()
    assert np.array_equal(got[0], want[0])
    c.check_attention()


@pytest.mark.parametrize("many,wide", [(25, False), (25, True), (700, False), (2100, False)])
@pytest.mark.parametrize("m", ["nan", "inf"])
def test_scores_that_are_nan_leave_the_first_and_last_pages(many, wide, m):
    c = Case(rows=[2], lens=[16 * many], page=16, heads=2, group=2, dim=64, top=5, first=1, last=2, wide=wide)
    c.bound_all()
    kind = np.zeros(64, np.int8)  # infinity times a sum of 0 is NaN
    for p in (3, 7, 9):
        for h in range(2):
            c.ref_bounds[c.table[0, p]].reshape(2, -1)[h] = select_ref.record_of(kind, kind, np.float32(m))
    c.bounds.copy_(torch.from_numpy(c.ref_bounds))
    pages, kept = c.select()
    assert np.array_equal(pages, np.broadcast_to(c.table[0][[0, 3, 7, many - 2, many - 1]], (2, 2, 5)))
    assert kept.tolist() == [79, 80]
    c.check_attention()


@pytest.mark.parametrize("wide", [False, True])
def test_a_step_on_another_stream(wide):
    c = Case(rows=[2, 1], lens=[400, 300], page=16, heads=2, group=2, dim=64, top=5, wide=wide)
    c.bound_all()
    torch.cuda.synchronize()
    s, out, q = torch.cuda.Stream(), torch.empty_like(c.q), c.q.clone()
    size = max(binding.dspark_kv4_select_workspace_bytes(c.cache, c.batch, c.selection),
               binding.dspark_kv4_attention_selected_workspace_bytes(c.cache, c.selection, 4))
    ws = c.scratch(size)
    c.q.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # the queries come late: on another stream the calls would not see them
        c.q.copy_(q)
    binding.dspark_kv4_bound_pages(c.cache, c.batch, c.bounds, stream=s)
    binding.dspark_kv4_select(c.cache, c.batch, c.bounds, c.q, c.selection, ws, first=c.first, last=c.last, stream=s)
    binding.dspark_kv4_attention_selected(c.cache, c.selection, c.q, out, c.scale, ws, stream=s)
    torch.cuda.synchronize()
    want = c.wanted()
    assert np.array_equal(c.pages.cpu().numpy(), want[0]) and np.array_equal(c.kept.cpu().numpy(), want[1])
    assert torch.equal(c.attend()[0], out)


@pytest.mark.parametrize("wide", [False, True])
def test_rows_of_no_request_and_strided_queries(wide):
    c = Case(rows=[3, 4], lens=[200, 90], page=16, heads=2, group=2, dim=64, top=3, wide=wide)
    c.bound_all()
    c.batch.tensors[0].copy_(ints([1, 2, 5]))
    pages, kept = c.select()
    assert kept.tolist()[0] == kept.tolist()[5] == kept.tolist()[6] == -1 and min(kept[1:5]) > 0
    out, lse = c.attend()
    assert (out[[0, 5, 6]] == -55).all() and (lse[[0, 5, 6]] == -55).all() and not (out[1:5] == -55).any()
    d = Case(rows=[3, 4], lens=[200, 90], page=16, heads=2, group=2, dim=64, top=3, wide=wide)
    d.bound_all()
    wide = torch.zeros(7, 4 * 64 + 1, dtype=d.q.dtype, device="cuda")
    view = wide[:, 1:].unflatten(1, (4, 64))
    view.copy_(d.q)
    a = d.select()[0].copy()
    d.pages.fill_(-3)
    b = d.select(q=view)[0]
    assert np.array_equal(a, b)


def test_rows_without_any_request():
    c = Case(rows=[3], lens=[200], page=16, heads=2, group=2, dim=64, top=3)
    c.batch = binding.Kv4Batch(ints([0]), ints([200]), ints(c.table), total_rows=3, max_rows=0, slots=ints([]))
    binding.dspark_kv4_bound_pages(c.cache, c.batch, c.bounds)
    pages, kept = c.select()
    assert (pages == -1).all() and (kept == -1).all()
    out, _ = c.attend()
    assert (out == -55).all()


@pytest.mark.parametrize("kw", [dict(rows=[1, 1, 1], lens=[333, 64, 1], page=64, heads=2, group=8, dim=128),
                                dict(rows=[1, 1], lens=[900, 40], page=16, heads=5, group=5, dim=64, dtype="f16")])
def test_all_pages_are_the_attention_of_the_cache(kw):
    """Both within the same bound of the same 64-bit values."""
    c = Case(top=80, **kw)
    c.check()
    pages, kept = c.select()
    for i in range(len(kw["rows"])):
        n = -(-kw["lens"][i] // kw["page"])
        assert (pages[i, :, :n] == c.table[i, :n]).all() and (pages[i, :, n:] == -1).all() and kept[i] == kw["lens"][i]
    want = select_ref.attention(c.ref, pages, kept, c.q.double().cpu().numpy(), c.group, c.scale)[0]
    whole = select_ref.kv4_ref.attention(c.ref, c.start, c.slots, c.lens, c.table, c.q.double().cpu().numpy(), c.group,
                                         c.scale, 0)[0]
    assert np.array_equal(want, whole)
    c.check_attention()


@pytest.mark.parametrize("wide", [False, True])
def test_more_rows_than_a_call_of_attention_takes(wide):
    c = Case(rows=[4200], lens=[4200], page=64, heads=1, group=1, dim=64, top=3, wide=wide)
    c.bound_all()
    pages, kept = c.select()
    rng = np.random.default_rng(0)
    some = np.concatenate([[0, 63, 64, 4095, 4096, 4097, 4199], rng.integers(0, 4200, 20)])
    q = c.q.float().cpu().numpy()
    for row in some:
        ids = select_ref.select(c.ref_bounds.reshape(c.ref.num_pages, 1, -1)[:, 0], c.ref.num_pages, 64, c.table[0], row,
                                q[row, :1], False, 64, 3, 1, 1)
        assert pages[row, 0, :len(ids)].tolist() == ids
    out, _ = c.attend()
    want, _, tol = select_ref.attention(c.ref, pages[some], kept[some], c.q.double().cpu().numpy()[some], 1, c.scale)
    got = out.double().cpu().numpy()[some]
    assert np.all(np.abs(got - want) <= 2 * (tol + 2.0 ** -9 * np.abs(want)) + 2.0 ** -24)


@pytest.mark.parametrize("wide", [False, True])
def test_many_requests(wide):
    n = 1000
    rng = np.random.default_rng(2)
    c = Case(rows=[1] * n, lens=[int(x) for x in rng.integers(0, 120, n)], page=16, heads=1, group=2, dim=64, top=3, wide=wide)
    for s in range(n):  # the reference's bounds, then all at once
        for p in range(-(-int(c.lens[s]) // 16)):
            c.put(s, p)
    c.bounds.copy_(torch.from_numpy(c.ref_bounds))
    got, want = c.select(), c.wanted()
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("group,dtype", [(64, "bf16"), (200, "f16")])
def test_wide_lists_and_large_groups(group, dtype):
    """Lists that could hold so much that the kernels of 128 and 256 rows are taken."""
    c = Case(rows=[2, 1], lens=[300, 40], page=16, heads=2, group=group, dim=64, top=30000, dtype=dtype)
    pages, kept = c.select()
    assert kept.tolist() == [299, 300, 40]
    for row, (slot, n) in enumerate(((0, 19), (0, 19), (1, 3))):
        assert (pages[row, :, :n] == c.table[slot, :n]).all() and (pages[row, :, n:] == -1).all()
    c.check_attention()


@pytest.mark.parametrize("wide", [False, True])
def test_captured_and_replayed(wide):
    c = Case(rows=[2, 1], lens=[400, 300], page=16, heads=2, group=2, dim=64, top=5, wide=wide)
    c.bound_all()
    q = c.q.clone()
    size = max(binding.dspark_kv4_select_workspace_bytes(c.cache, c.batch, c.selection),
               binding.dspark_kv4_attention_selected_workspace_bytes(c.cache, c.selection, 4))
    ws, out = c.scratch(size), torch.empty_like(q)

    def step():
        binding.dspark_kv4_bound_pages(c.cache, c.batch, c.bounds)
        binding.dspark_kv4_select(c.cache, c.batch, c.bounds, c.q, c.selection, ws)
        binding.dspark_kv4_attention_selected(c.cache, c.selection, c.q, out, c.scale, ws)
    c.first, c.last = 1, 2
    c.q.zero_()
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    c.q.copy_(q)
    graph.replay()
    torch.cuda.synchronize()
    want = c.wanted()
    assert np.array_equal(c.pages.cpu().numpy(), want[0]) and np.array_equal(c.kept.cpu().numpy(), want[1])
    again, _ = c.attend()
    assert torch.equal(again, out)
