"""Attention over the paged 4-bit cache against the 64-bit restatement of
tests/kv4_ref.py, within the bound derived there (and the output type's
rounding: 2^-9 for BF16, 2^-12 for FP16, doubled for the bound's first order)."""
import numpy as np
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests import kv4_ref
from tests.test_gpu_kv4_cache import TYPES, ints

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, rows, lens, page, heads, group, dim, *, dtype="bf16", window=0, gk=None, gv=None, slots=None,
                 seed=0, peak=1.0, scale=None, normal=True, table=None, wide=False):
        rng = np.random.default_rng(seed)
        self.rows, self.heads, self.group, self.dim, self.window, self.dtype = rows, heads, group, dim, window, dtype
        self.start = np.concatenate([[0], np.cumsum(rows)]).astype(int)
        self.total = int(self.start[-1])
        self.slots = list(range(len(rows))) if slots is None else slots
        self.lens = np.zeros(max([s for s in self.slots if s < 1000] + [0]) + 2, int)
        for s, n in zip(self.slots, lens):
            if s < 1000:
                self.lens[s] = n
        need = [-(-n // page) for n in self.lens]
        num_pages = sum(need) + 3
        ids = rng.permutation(num_pages)
        # what page tables can hold has a part in the choice of kernel: wide ones make every call a large one
        self.table = np.full((len(self.lens), 30000 if wide else max(max(need), 1)), -1)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = ids[at:at + n]
            at += n
        if table:
            table(self.table, num_pages)
        self.ref = kv4_ref.Cache(num_pages, page, heads, dim, gk, gv, rng)
        if normal:  # what append would leave, in pages of their own; the bytes behind a length stay random
            x = rng.standard_normal((2, num_pages, heads, page, dim))
            for w in range(2):
                code, scale_b = kv4_ref.quantise(x[w], 1.0)
                half, eighth = page * dim // 2, page * dim // 16
                r = self.ref.data.reshape(num_pages, heads, -1)
                r[:, :, w * half:(w + 1) * half] = (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(
                    num_pages, heads, -1)
                r[:, :, 2 * half + w * eighth:2 * half + (w + 1) * eighth] = scale_b.reshape(num_pages, heads, -1)
        f32 = lambda g: None if g is None else torch.tensor(g, dtype=torch.float32, device="cuda")  # noqa: E731
        self.data = torch.from_numpy(self.ref.data).cuda()
        self.cache = binding.Kv4Cache(self.data, page, heads, dim, k_scale=f32(gk), v_scale=f32(gv))
        self.batch = binding.Kv4Batch(ints(self.start), ints(self.lens), ints(self.table), total_rows=self.total,
                                      max_rows=max(rows), slots=None if slots is None else ints(slots))
        self.q = torch.from_numpy(peak * rng.standard_normal((self.total, heads * group, dim))).to(TYPES[dtype]).cuda()
        self.scale = dim ** -0.5 if scale is None else scale

    def workspace(self):
        n = binding.dspark_kv4_attention_workspace_bytes(self.cache, self.batch, self.heads * self.group)
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN everywhere

    def run(self, lse=True, q=None, out=None):
        q = self.q if q is None else q
        out = torch.full_like(self.q, -55.0) if out is None else out
        lse = torch.full((self.total, self.heads * self.group), -55.0, device="cuda") if lse else None
        binding.dspark_kv4_attention(self.cache, self.batch, q, out, self.scale, self.workspace(), window=self.window,
                                     lse=lse)
        torch.cuda.synchronize()
        return out, lse

    def check(self, **kw):
        out, lse = self.run(**kw)
        want, want_lse, tol = kv4_ref.attention(self.ref, self.start, self.slots, self.lens, self.table,
                                                self.q.double().cpu().numpy(), self.group, self.scale, self.window)
        got = out.double().cpu().numpy()
        unit = 2.0 ** -9 if self.dtype == "bf16" else 2.0 ** -12
        room = 2 * (tol + unit * np.abs(want)) + 2.0 ** -24
        assert np.all(np.abs(got - want) <= room), np.max(np.abs(got - want) / room)
        if lse is not None:
            got = lse.double().cpu().numpy()
            empty = np.isneginf(want_lse)
            assert np.array_equal(np.isneginf(got), empty)
            # log of a sum of weights that are off by a share d: off by d
            d = 2.0 ** -20 * (1 + np.abs(want_lse[~empty])) + tol[~empty].max(initial=0)
            assert np.all(np.abs(got[~empty] - want_lse[~empty]) <= d)
        return out


CASES = [
    dict(rows=[1], lens=[1], page=16, heads=1, group=1, dim=64),
    dict(rows=[1], lens=[64], page=64, heads=1, group=8, dim=128),
    dict(rows=[1, 1, 1, 1], lens=[63, 64, 65, 1000], page=64, heads=2, group=4, dim=128),
    dict(rows=[1, 1, 1], lens=[15, 16, 17], page=16, heads=3, group=5, dim=64, dtype="f16"),
    dict(rows=[6, 6], lens=[6, 300], page=32, heads=2, group=8, dim=128),
    dict(rows=[6, 1, 0, 3], lens=[129, 127, 50, 2], page=128, heads=1, group=2, dim=128),   # 3 rows, 2 tokens
    dict(rows=[2, 2], lens=[700, 0], page=256, heads=2, group=7, dim=64),                   # an empty cache
    dict(rows=[17, 40], lens=[17, 90], page=16, heads=2, group=3, dim=128, dtype="f16"),
    dict(rows=[1, 5], lens=[500, 333], page=64, heads=1, group=16, dim=128, window=1),
    dict(rows=[9, 1], lens=[400, 333], page=32, heads=1, group=4, dim=64, window=100),
    dict(rows=[6, 6], lens=[200, 64], page=64, heads=2, group=8, dim=128, window=64, dtype="f16"),
    dict(rows=[1, 2], lens=[100, 77], page=16, heads=2, group=2, dim=128, gk=[0.03, 2.5], gv=[0.4, 1.7]),
    dict(rows=[3, 1, 2], lens=[50, 20, 90], page=32, heads=2, group=1, dim=64, slots=[5, 0, 2]),
    dict(rows=[150], lens=[333], page=64, heads=1, group=8, dim=128),                       # many tiles
    dict(rows=[130, 7], lens=[130, 900], page=16, heads=1, group=5, dim=64, window=77, dtype="f16"),
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kw", CASES)
def test_against_64_bits(kw, wide):
    Case(wide=wide, **kw).check()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
def test_peaked_and_flat_weights(dim, wide):
    """One key far above the others; all scores equal (scale 0); a negative scale."""
    for peak, scale in ((12.0, None), (1.0, 0.0), (1.0, -0.2)):
        Case([2, 1], [300, 70], 64, 2, 4, dim, peak=peak, scale=scale, seed=3, wide=wide).check()
        Case([40, 1], [300, 70], 64, 1, 4, dim, peak=peak, scale=scale, seed=3, wide=wide).check()


@pytest.mark.parametrize("rows", [4, 30])
@pytest.mark.parametrize("wide", [False, True])
def test_any_bytes_are_finite_numbers(rows, wide):
    """Random bytes, NaN scales among them, wherever a row may see them or not: no NaN gets out, and what a row
    may not see has no part in it."""
    c = Case([rows, 1], [100, 200], 16, 2, 4, 64, normal=False, scale=1e-6, seed=9, wide=wide)
    out, lse = c.run()
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    c.check()
    # tokens behind the length, and pages of others
    first = c.run()[0].clone()
    data = c.data.cpu().numpy()
    for s in (0, 1):
        last = c.table[s, -(-c.lens[s] // 16) - 1]
        keep = c.lens[s] % 16 or 16
        r = data[last].reshape(2, -1)
        for w, (at, n) in enumerate(((0, 32), (16 * 32, 32), (2 * 16 * 32, 4), (2 * 16 * 32 + 16 * 4, 4))):
            r[:, at + keep * n:at + 16 * n] = 0x7F
    c.data.copy_(torch.from_numpy(data))
    assert torch.equal(first, c.run()[0])


def test_pages_that_are_not_there():
    def holes(table, num_pages):
        table[0, 1], table[0, 3], table[1, 0] = -1, num_pages, 10 ** 8
    for page in (16, 32, 64, 128):
        for rows in ([2, 3], [9, 20], [80, 3]):
            Case(rows, [6 * page + 5, 2 * page], page, 1, 4, 128, table=holes, seed=page, wide=True).check()
        Case([2, 3], [6 * page + 5, 2 * page], page, 1, 4, 128, table=holes, seed=page).check()

    def none(table, num_pages):
        table[:] = -5
    out = Case([2], [100], 32, 1, 4, 64, table=none).check()
    assert not out.any()


def test_requests_that_are_not_there_and_rows_of_nobody():
    c = Case([2, 2, 1], [70, 70, 40], 64, 1, 4, 64, slots=[1, 5000, 0])
    out, lse = c.run()
    assert not out[2:4].any() and torch.isneginf(lse[2:4]).all()
    c.check()
    start = ints([1, 2, 3, 4])
    c.batch = binding.Kv4Batch(start, ints(c.lens), ints(c.table), total_rows=5, max_rows=2, slots=ints([1, 1, 0]))
    out, _ = c.run()
    assert torch.all(out[0] == -55.0) and torch.all(out[4] == -55.0)


@pytest.mark.parametrize("wide", [False, True])
def test_strided_queries_and_outputs(wide):
    c = Case([6, 1], [100, 33], 64, 2, 4, 128, wide=wide)
    want, _ = c.run()
    for offset in (0, 8, 1):
        wide = torch.zeros(c.total, 12 * 128 + 16 + offset, dtype=torch.bfloat16, device="cuda")
        q = wide[:, offset:offset + 8 * 128].unflatten(1, (8, 128))
        q.copy_(c.q)
        place = torch.full_like(wide, 3.0)
        out = place[:, offset:offset + 8 * 128].unflatten(1, (8, 128))
        got, _ = c.run(q=q, out=out)
        assert torch.equal(got, want)
        assert torch.all(place[:, :offset] == 3.0) and torch.all(place[:, offset + 8 * 128:] == 3.0)


@pytest.mark.parametrize("rows", [3, 10, 50])
def test_a_large_query_range(rows):
    """BF16 queries whose values FP16 cannot hold: rows of 1e30 and of 1e-30 (with scales that bring the scores
    back) and rows with a wide spread."""
    for size, scale in ((1e30, 1e-31), (1e-30, 1e29)):
        c = Case([rows], [90], 64, 1, 4, 128, scale=scale, wide=True)
        c.q.mul_(size)
        c.check()
    c = Case([rows], [90], 64, 1, 4, 128, wide=True)
    c.q[..., ::7] *= 2.0 ** -20
    c.check()


def on_gpu(c):
    """What kv4_ref.attention gives, in FP64 on the GPU from the values that dspark_kv4_read gives (exact in FP32)."""
    out = torch.zeros(c.total, c.heads * c.group, c.dim, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    u = 2.0 ** -24
    for i, slot in enumerate(c.slots):
        n, rows = int(c.lens[slot]), c.rows[i]
        if n == 0 or rows == 0:
            continue
        k = torch.empty(n, c.heads, c.dim, device="cuda")
        v = torch.empty_like(k)
        whole = binding.Kv4Batch(ints([0, n]), ints(c.lens), ints(c.table), total_rows=n, max_rows=n,
                                 slots=ints([slot]))
        binding.dspark_kv4_read(c.cache, whole, k, v)
        q = c.q[c.start[i]:c.start[i + 1]].double().unflatten(1, (c.heads, c.group))
        pos = torch.arange(rows, device="cuda") + n - rows
        key = torch.arange(n, device="cuda")
        seen = key <= pos[:, None]
        if c.window:
            seen &= key > pos[:, None] - c.window
        for h in range(c.heads):
            ks, vs = k[:, h].double(), v[:, h].double()
            for g in range(c.group):
                x = q[:, h, g]
                s = (x @ ks.T * c.scale).masked_fill(~seen, -torch.inf)
                top = s.amax(1, keepdim=True)
                top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
                w = torch.exp(s - top)
                low = w.sum(1, keepdim=True)
                some = low > 0
                low = torch.where(some, low, torch.ones_like(low))
                size = (x.abs() @ ks.abs().T * abs(c.scale)).masked_fill(~seen, 0).amax(1, keepdim=True)
                spread = torch.where(seen, (s - top).abs(), torch.zeros_like(s)).amax(1, keepdim=True)
                d = (c.dim + 6) * u * size + 2.0 ** -20 + 4 * u * spread + (n / 16 + 16) * u
                at = slice(c.start[i], c.start[i + 1]), h * c.group + g
                out[at] = w @ vs / low
                tol[at] = (2.0 ** -11 + 2 * d) * (w @ vs.abs()) / low + 2.0 ** -29 * (seen.double() @ vs.abs())
    return out, tol


LONG = [
    dict(rows=[1, 1, 2, 1, 1], lens=[20000, 1, 7000, 64, 12345], page=64, heads=2, group=8, dim=64),    # tiles of 16 rows
    dict(rows=[1, 1], lens=[30001, 9000], page=32, heads=1, group=8, dim=128, dtype="f16"),             # of 8 rows
    dict(rows=[6, 6, 1], lens=[5000, 3, 777], page=64, heads=2, group=8, dim=128),                      # of 128 rows
    dict(rows=[8, 8, 5, 1], lens=[4097, 64, 9001, 1], page=128, heads=1, group=16, dim=64),
    dict(rows=[300], lens=[5000], page=32, heads=1, group=4, dim=128),                                  # of 256 rows
    dict(rows=[257, 1, 60], lens=[6001, 4000, 61], page=256, heads=2, group=2, dim=128, dtype="f16"),
    dict(rows=[200, 50, 0, 7], lens=[3333, 2000, 9, 3], page=16, heads=2, group=5, dim=64, dtype="f16", window=700),
    dict(rows=[40, 3], lens=[4000, 4000], page=64, heads=1, group=7, dim=128, window=100, scale=0.5),
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kw", LONG)
def test_runs_of_blocks_that_cut_units(kw, wide):
    """Enough blocks that units are cut by the CTAs' runs in many ways; the same call twice gives the same bits."""
    c = Case(seed=4, wide=wide, **kw)
    a, _ = c.run()
    b, _ = c.run()
    assert torch.equal(a, b)
    want, tol = on_gpu(c)
    unit = 2.0 ** -9 if c.dtype == "bf16" else 2.0 ** -12
    room = 2 * (tol + unit * want.abs()) + 2.0 ** -24
    assert ((a.double() - want).abs() <= room).all(), ((a.double() - want).abs() / room).max()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("most", [1, 2, 9, 40])
def test_many_short_units(most, wide):
    """Hundreds of requests of none to three blocks, some without rows or tokens: runs that hold many units, start in
    front of a unit's first block and end behind another's last."""
    rng = np.random.default_rng(most)
    rows = [int(n) for n in rng.integers(0, most + 1, 300)] + [most]
    lens = [int(n) * int(k) for n, k in zip(rng.integers(0, 150, 301), rng.random(301) > 0.1)]
    c = Case(rows, lens, 32, 3, 8, 64, seed=most, wide=wide)
    out, _ = c.run()
    want, tol = on_gpu(c)
    room = 2 * (tol + 2.0 ** -9 * want.abs()) + 2.0 ** -24
    assert ((out.double() - want).abs() <= room).all(), ((out.double() - want).abs() / room).max()


@pytest.mark.parametrize("kw", LONG[4:])
def test_more_rows_than_promised(kw):
    """max_rows chooses the kernel only: the kernels of few rows compute requests of many."""
    c = Case(seed=5, wide=True, **kw)
    want, tol = on_gpu(c)
    unit = 2.0 ** -9 if c.dtype == "bf16" else 2.0 ** -12
    for promised in (1, 16 // c.group, 128 // c.group):
        c.batch = binding.Kv4Batch(ints(c.start), ints(c.lens), ints(c.table), total_rows=c.total, max_rows=promised)
        out, _ = c.run()
        room = 2 * (tol + unit * want.abs()) + 2.0 ** -24
        assert ((out.double() - want).abs() <= room).all(), promised


def test_a_row_of_nan_stays_alone():
    """A query row with NaN or an infinity is NaN; the rows beside it are as without it."""
    for rows in (1, 6, 40):
        c = Case([rows, rows], [300, 200], 64, 1, 8, 128, seed=rows, wide=True)
        want, _ = c.run()
        c.q[0, 3, 5] = float("nan")
        c.q[rows, 2, 7] = float("inf")
        out, _ = c.run()
        bad = torch.isnan(out.float()).any(2)
        assert bad[0, 3] and bad[rows, 2] and bad.sum() == 2
        assert torch.equal(out[~bad], want[~bad])


def test_another_stream_and_a_graph():
    c = Case([6, 1], [300, 33], 64, 2, 8, 128)
    want, _ = c.run()
    out, work = torch.zeros_like(c.q), c.workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        binding.dspark_kv4_attention(c.cache, c.batch, c.q, out, c.scale, work)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.dspark_kv4_attention(c.cache, c.batch, c.q, out, c.scale, work)
    out.zero_()
    c.q.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, c.run()[0]) and not torch.equal(out, want)


def test_refusals():
    c = Case([2], [40], 16, 2, 2, 64)
    out, work = torch.empty_like(c.q), c.workspace()

    def code(**kw):
        try:
            a = dict(q=c.q, out=out, scale=1.0, workspace=work, window=0)
            a.update(kw)
            binding.dspark_kv4_attention(c.cache, c.batch, a["q"], a["out"], a["scale"], a["workspace"],
                                         window=a["window"])
        except binding.DsparkError as e:
            return e.code
        return 0
    assert code() == 0
    assert code(window=-1) == -1
    assert code(scale=float("nan")) == -1 and code(scale=float("inf")) == -1
    assert code(workspace=work[:-256]) == -1
    assert code(workspace=work[16:]) in (-1, -3)
    assert code(q=c.q[:, :3], out=out[:, :3]) == -1   # not a multiple of the key/value heads
    with pytest.raises(TypeError):
        code(q=c.q.half())
    with pytest.raises(ValueError):
        code(q=c.q[:, :, :32], out=out[:, :, :32])
