"""The token table and the adjusted logits (include/dspark_logits.h).  Counts and marks are whole numbers.  A logit is
up to six FP32 operations, each rounded once: the same operations in numpy give the same bits; and from the formula in
64 bits it is off by at most 2^-24 of each operation's result, and half a step of the output's type."""
import numpy as np
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding

pytestmark = pytest.mark.gpu
F = np.float32
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def bits(flags):
    """Truth values [..., n] as int32 words."""
    n = flags.shape[-1]
    f = np.zeros((*flags.shape[:-1], -(-n // 32) * 32), bool)
    f[..., :n] = flags
    return np.packbits(f, axis=-1, bitorder="little").view(np.int32)


class Table:
    def __init__(self, slots, vocab, pad=0):
        words = -(-vocab // 32)
        wide = torch.zeros(slots, vocab + pad, dtype=torch.int32, device="cuda")
        marks = torch.zeros(slots, 2 + (pad > 0), words, dtype=torch.int32, device="cuda")
        self.wide, self.wide_marks = wide, marks
        self.counts, self.marks = wide[:, :vocab], marks[:, :2]
        self.table = binding.TokenTable(self.counts, self.marks)
        self.want = np.zeros((slots, vocab), np.int64)
        self.prompt = np.zeros((slots, vocab), bool)
        self.vocab, self.slots = vocab, slots

    def count(self, tokens, lens, slots=None, prompt=False, reset=False, kind=torch.int64):
        t = torch.from_numpy(np.asarray(tokens)).to(kind).cuda()
        binding.dspark_tokens_count(self.table, t, ints(lens), slots=None if slots is None else ints(slots),
                                    prompt=prompt, reset=reset)
        at = range(len(lens)) if slots is None else slots
        for s in at:
            if reset and 0 <= s < self.slots:
                self.want[s], self.prompt[s] = 0, False
        for i, s in enumerate(at):
            if not 0 <= s < self.slots:
                continue
            for v in np.asarray(tokens)[i][:max(0, min(lens[i], np.shape(tokens)[1]))]:
                if 0 <= v < self.vocab:
                    if prompt:
                        self.prompt[s, v] = True
                    else:
                        self.want[s, v] += 1

    def check(self):
        assert np.array_equal(self.counts.cpu().numpy(), self.want)
        assert np.array_equal(self.marks.cpu().numpy(), bits(np.stack([self.prompt, self.want > 0], 1)))


@pytest.mark.parametrize("vocab,slots,pad", [(1, 1, 0), (31, 3, 0), (32, 2, 0), (33, 5, 3), (5000, 4, 0), (129281, 2, 7)])
def test_counts_and_marks(vocab, slots, pad):
    rng = np.random.default_rng(vocab)
    t = Table(slots, vocab, pad)
    some = [int(x) for x in rng.integers(0, slots, 3)]  # a slot may come twice
    skewed = lambda n, w: (rng.random((n, w)) ** 4 * (vocab + 1)).astype(np.int64) - (rng.random((n, w)) < 0.01)  # noqa: E731
    t.count(skewed(3, 700), [700, 0, 650], some, prompt=True, reset=True)
    t.count(skewed(3, 300), [-4, 1000, 17], some)
    t.check()
    t.count(skewed(slots, 9), [9] * slots, kind=torch.int32)
    t.count(skewed(3, 5), [5, 5, 5], [slots, -1, 0], prompt=True, kind=torch.int32)
    t.check()
    t.count(skewed(2, 1000), [1000, 3], [0, slots - 1], reset=True)
    t.check()
    if pad:
        assert (t.wide[:, vocab:] == 0).all() and (t.wide_marks[:, 2] == 0).all()


def test_reset_clears_what_a_table_held_before_and_nothing_else():
    t = Table(4, 1001, 5)
    t.wide.fill_(9)
    t.wide_marks.fill_(-1)
    empty = np.zeros((2, 0), np.int64)
    t.count(empty, [0, 0], [2, 0], reset=True)
    assert (t.counts[[0, 2]] == 0).all() and (t.marks[[0, 2]] == 0).all()
    assert (t.counts[[1, 3]] == 9).all() and (t.marks[[1, 3]] == -1).all()
    assert (t.wide[:, 1001:] == 9).all() and (t.wide_marks[:, 2] == -1).all()


@pytest.mark.parametrize("width", [5, 5000])
def test_cleared_before_what_follows_where_there_are_no_tokens(width):
    """Nothing is counted, so nothing else waits for the slots to be cleared."""
    t = Table(200, 129280)
    ids = torch.zeros(200, width, dtype=torch.int64, device="cuda")
    none, slots = ints([0] * 200), ints(list(range(200)))
    for _ in range(5):
        t.wide.fill_(3)
        t.wide_marks.fill_(-1)
        binding.dspark_tokens_count(t.table, ids, none, slots=slots, reset=True)
        left = t.wide.amax(1) + t.wide_marks.flatten(1).abs().amax(1)
        assert (left == 0).all()


def test_a_long_history():
    rng = np.random.default_rng(7)
    t = Table(1, 300, 0)
    tokens = rng.integers(0, 300, (1, 130000)) % 250
    binding.dspark_tokens_count(t.table, torch.from_numpy(tokens).cuda(), ints([130000]))
    t.want[0] = np.bincount(tokens[0], minlength=300)
    t.check()


@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_many_long_lists(prompt, kind):
    """Enough tokens for the kernel that marks in shared memory; slots listed twice, lists of every length."""
    rng = np.random.default_rng(11)
    t = Table(40, 5001, 3)
    lens = [20000, 0, 1, 8191, 8192, 8193, 16384, 50000, -3] + [int(x) for x in rng.integers(0, 20001, 31)]
    slots = [int(x) for x in rng.permutation(40)]
    slots[5], slots[20], slots[21] = slots[7], 40, -1
    tokens = ((rng.random((40, 20000)) ** 3) * 5003).astype(np.int64) - 1
    ids = torch.from_numpy(tokens).to(kind).cuda()
    t.wide[slots[0]] = 7
    t.wide_marks[slots[0], :2] = -1
    for reset in (True, False):
        binding.dspark_tokens_count(t.table, ids, ints(lens), slots=ints(slots), prompt=prompt, reset=reset)
        for i, s in enumerate(slots):
            if 0 <= s < 40:
                here = tokens[i][:max(0, min(lens[i], 20000))]
                n = np.bincount(here[(here >= 0) & (here < 5001)], minlength=5001)
                if prompt:
                    t.prompt[s] |= n > 0
                else:
                    t.want[s] += n
    t.check()
    assert (t.wide_marks[:, 2] == 0).all()


class Case:
    def __init__(self, batch, drafts, vocab, *, dtype="bf16", out="f32", slots=None, max_slots=None, held=20, seed=0,
                 repetition=True, frequency=True, presence=True, bias=3, mask="rows", table=True, spread=3.0):
        rng = np.random.default_rng(seed)
        self.batch, self.drafts, self.vocab, self.out_type = batch, drafts, vocab, TYPES[out]
        self.slots = slots
        self.n = max_slots or batch
        self.rows = batch * (drafts + 1)
        self.logits = torch.from_numpy(rng.standard_normal((self.rows, vocab)) * spread).to(TYPES[dtype]).cuda()
        self.t = Table(self.n, vocab) if table else None
        if table:
            self.t.count(rng.integers(0, vocab, (self.n, held)), [held] * self.n, prompt=True)
            self.t.count(rng.integers(0, vocab, (self.n, held)) // 3, [held] * self.n)
        self.draft = rng.integers(-1, vocab + 1, (batch, drafts)) if drafts else None
        if drafts > 1:
            self.draft[:, -1] = self.draft[:, 0]
        pen = lambda on, lo, hi: rng.uniform(lo, hi, self.n).astype(F) if on else None  # noqa: E731
        self.pen = dict(repetition=pen(repetition, 0.8, 1.5), frequency=pen(frequency, -0.4, 0.7),
                        presence=pen(presence, 0.0, 0.5))
        self.bias = None
        if bias:
            count = rng.integers(0, 2 * bias + 1, self.n)
            start = np.concatenate([[0], np.cumsum(count)])
            ids = rng.integers(-1, vocab + 1, start[-1])
            for s in range(self.n):  # one id twice
                if count[s] > 1:
                    ids[start[s + 1] - 1] = ids[start[s]]
            self.bias = (start, ids, rng.standard_normal(start[-1]).astype(F))
        self.mask = self.mask_rows = None
        if mask:
            self.mask = rng.random((self.rows, vocab)) < rng.choice([0.02, 0.5, 0.98], (self.rows, 1))
            self.mask[0] = False
            if mask == "picked":
                self.mask_rows = rng.integers(-1, self.rows + 1, self.rows)

    def arguments(self):
        f32 = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
        a = {k: f32(v) for k, v in self.pen.items()}
        if self.bias is not None:
            a["bias"] = (ints(self.bias[0]), ints(self.bias[1]), f32(self.bias[2]))
        if self.mask is not None:
            a["mask"] = torch.from_numpy(bits(self.mask)).cuda()
        if self.mask_rows is not None:
            a["mask_rows"] = ints(self.mask_rows)
        if self.slots is not None:
            a["slots"] = ints(self.slots)
        if self.draft is not None:
            a["draft"] = torch.from_numpy(self.draft).cuda()
        return dict(a, drafts=self.drafts, max_slots=self.n)

    def run(self, logits=None, out=None):
        logits = self.logits if logits is None else logits
        out = torch.full(logits.shape, -55.0, dtype=self.out_type, device="cuda") if out is None else out
        binding.dspark_logits_adjust(self.t and self.t.table, logits, out, **self.arguments())
        torch.cuda.synchronize()
        return out

    def wanted(self, kind):
        """In numpy's type `kind`; and in 64 bits how far FP32's roundings can be from it."""
        x = self.logits.float().cpu().numpy().astype(kind)
        room = np.zeros(x.shape)
        u = 2.0 ** -24
        for r in range(self.rows):
            i, j = divmod(r, self.drafts + 1)
            s = i if self.slots is None else self.slots[i]
            l = x[r]  # noqa: E741
            if 0 <= s < self.n:
                n = np.zeros(self.vocab, np.int64) if self.t is None else self.t.want[s].copy()
                if self.draft is not None:
                    for v in self.draft[i][:j]:
                        if 0 <= v < self.vocab:
                            n[v] += 1
                prompt = np.zeros(self.vocab, bool) if self.t is None else self.t.prompt[s]
                rep, freq, pres = (None if p is None else kind(p[s]) for p in self.pen.values())
                if rep is not None:
                    l = np.where((n > 0) | prompt, np.where(l > 0, l / rep, l * rep), l).astype(kind)
                    room[r] += u * np.abs(l)
                if freq is not None:
                    by = (freq * n.astype(kind)).astype(kind)
                    l = np.where(n > 0, l - by, l).astype(kind)
                    room[r] += u * (np.abs(by) + np.abs(l))
                if pres is not None:
                    l = np.where(n > 0, l - pres, l).astype(kind)
                    room[r] += u * np.abs(l)
                if self.bias is not None:
                    b = np.zeros(self.vocab, kind)
                    for e in range(self.bias[0][s], self.bias[0][s + 1]):
                        v = self.bias[1][e]
                        if 0 <= v < self.vocab:
                            b[v] += kind(self.bias[2][e])
                            room[r, v] += u * abs(b[v])
                    l = (l + b).astype(kind)
                    room[r] += u * np.abs(l)
            if self.mask is not None:
                m = r if self.mask_rows is None else self.mask_rows[r]
                if 0 <= m < len(self.mask):
                    l = np.where(self.mask[m], l, kind(-np.inf))
            x[r] = l
        return x, room

    def check(self, **kw):
        got = self.run(**kw)
        want = torch.from_numpy(self.wanted(F)[0]).to(self.out_type)
        assert torch.equal(got.cpu().nan_to_num(nan=1e30), want.nan_to_num(nan=1e30))
        exact, room = self.wanted(np.float64)
        got = got.double().cpu().numpy()
        half = 2.0 ** -8 if self.out_type == torch.bfloat16 else 0.0
        some = np.isfinite(exact)
        with np.errstate(invalid="ignore"):
            # twice: each rounding is relative to a value that is itself off, and a repetition multiplies what is
            room *= 2
            assert np.all((np.abs(got - exact) <= room + half * (np.abs(exact) + room) + 2.0 ** -140)[some])
        return got


CASES = [
    dict(batch=1, drafts=0, vocab=1, held=1, bias=1),
    dict(batch=1, drafts=0, vocab=2048),
    dict(batch=3, drafts=5, vocab=5000, out="bf16"),
    dict(batch=3, drafts=5, vocab=5003),
    dict(batch=2, drafts=1, vocab=4097, dtype="f32", mask="picked"),
    dict(batch=4, drafts=3, vocab=6144 + 40, dtype="f32", slots=[5, 1, -1, 9], max_slots=7),
    dict(batch=5, drafts=2, vocab=33, held=3, slots=[4, 4, 0, 1, 2], mask="picked"),  # a slot in two requests
    dict(batch=2, drafts=6, vocab=4096, mask=None, bias=0),
    dict(batch=2, drafts=6, vocab=4096, repetition=False, presence=False),
    dict(batch=2, drafts=3, vocab=4096, frequency=False, presence=False, out="bf16"),
    dict(batch=2, drafts=0, vocab=9000, repetition=False, frequency=False, presence=False),
    dict(batch=2, drafts=4, vocab=3000, table=False, mask="picked"),
    dict(batch=1, drafts=40, vocab=64, held=3, bias=300),
    dict(batch=1, drafts=1023, vocab=40, held=3, mask=None),
    dict(batch=300, drafts=0, vocab=100, held=7),
]


@pytest.mark.parametrize("kw", CASES)
def test_against_the_formula(kw):
    Case(**kw).check()


@pytest.mark.parametrize("kw", [dict(dtype="f32", out="f32"), dict(dtype="bf16", out="bf16")])
@pytest.mark.parametrize("vocab", [4096, 4097])
@pytest.mark.parametrize("mask", [None, "rows", "picked"])
def test_in_place(kw, vocab, mask):
    c = Case(3, 4, vocab, mask=mask, **kw)
    want = c.run()
    x = c.logits.clone()
    c.run(logits=x, out=x)
    assert torch.equal(x, want)


def test_rows_apart_and_unaligned():
    for pad, shift in ((8, 0), (8, 8), (5, 3)):
        c = Case(2, 2, 4000, dtype="bf16", out="bf16")
        wide = torch.zeros(c.rows, 4000 + pad + shift, dtype=torch.bfloat16, device="cuda")
        view = wide[:, shift:shift + 4000]
        view.copy_(c.logits)
        c.check(logits=view)
        c.check(logits=view, out=view)
        assert (wide[:, shift + 4000:] == 0).all() and (wide[:, :shift] == 0).all()


@pytest.mark.parametrize("kinds", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("vocab,drafts", [(1, 2), (6, 9), (9, 1), (509, 3), (512, 10), (517, 0), (1030, 36), (5003, 6)])
@pytest.mark.parametrize("shift,apart", [(3, 0), (8, 1), (5, 6), (1, 8), (7, 3)])
def test_rows_apart_from_the_same_unaligned_place(kinds, vocab, drafts, shift, apart):
    """Both sides' rows `vocab + apart` apart, from the same unaligned place on."""
    c = Case(2, drafts, vocab, dtype=kinds[0], out=kinds[1], held=min(vocab, 5), bias=min(vocab, 3), mask="rows")
    size = c.rows * (vocab + apart) + shift + 8
    x = torch.full((size,), -7.0, dtype=c.logits.dtype, device="cuda")
    y = torch.full((size,), -9.0, dtype=c.out_type, device="cuda")
    logits, out = (t.as_strided((c.rows, vocab), (vocab + apart, 1), shift) for t in (x, y))
    logits.copy_(c.logits)
    c.check(logits=logits, out=out)
    out.fill_(-9.0)
    assert (y == -9.0).all()  # nothing beside the rows


def test_masks_and_biases_alone_need_no_drafts():
    c = Case(2, 3, 3000, repetition=False, frequency=False, presence=False)
    want = c.run()
    c.draft = None
    assert torch.equal(c.run(), want)
    c = Case(2, 3, 3000, frequency=False)
    c.draft = None
    with pytest.raises(binding.DsparkError):
        c.run()


def test_infinities_and_nan():
    c = Case(2, 3, 3000, dtype="f32", mask="picked")
    for i, v in enumerate((float("inf"), float("-inf"), float("nan"), 0.0, -0.0, 3e38, -3e38, 1e-40)):
        c.logits[:, i::50] = v
    c.bias[2][::3] = -np.inf
    got = c.run().cpu().numpy()
    with np.errstate(all="ignore"):
        want = c.wanted(F)[0]
    assert np.array_equal(got, want, equal_nan=True)


def test_captured_and_replayed_with_what_was_said_since():
    c = Case(3, 2, 4000, mask=None)
    out = torch.empty(c.rows, 4000, device="cuda")
    a = c.arguments()
    binding.dspark_logits_adjust(c.t.table, c.logits, out, **a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.dspark_logits_adjust(c.t.table, c.logits, out, **a)
    c.t.count(np.arange(30).reshape(3, 10), [10, 3, 0])
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), c.wanted(F)[0])


def test_on_another_stream():
    c = Case(3, 2, 4000)
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    a = c.arguments()
    s.wait_stream(torch.cuda.current_stream())
    binding.dspark_logits_adjust(c.t.table, c.logits, out, stream=s, **a)
    s.synchronize()
    assert torch.equal(out, want)


def test_into_the_accept():
    """Adjusted BF16 logits and the greedy accept: a mask that allows one token makes it the answer."""
    b, p, v = 4, 3, 4096
    c = Case(b, p, v, dtype="bf16", out="bf16", mask=None)
    c.mask = np.ones((c.rows, v), bool)
    only = np.random.default_rng(1).integers(0, v, (b, p + 1))
    for r in range(c.rows):
        c.mask[r] = False
        c.mask[r, only.reshape(-1)[r]] = True
    out = c.run()
    draft = torch.from_numpy(only[:, :p].copy()).cuda()
    draft[0, 1] = (draft[0, 1] + 1) % v
    accepted = torch.empty(b, p + 1, dtype=torch.int64, device="cuda")
    count = torch.empty(b, dtype=torch.int32, device="cuda")
    binding.dspark_greedy_accept_noalloc(out, draft, ints([p] * b), accepted, count, b, p, p, v)
    assert count.tolist() == [2] + [p + 1] * (b - 1)
    assert accepted[1:].cpu().numpy().tolist() == only[1:].tolist()
    binding.dspark_tokens_count(c.t.table, accepted, count)
    for i in range(b):
        for x in only[i][:count.tolist()[i]]:
            c.t.want[i, x] += 1
    c.t.check()
