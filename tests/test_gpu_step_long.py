"""The loops of kernels whose warps and CTAs stay: steps with so much to do that each takes several items in turn, with
another request's in between.  adjust_kernel has 3040 warps (2432 where rows are not aligned) and units of 512 tokens,
score_kernel 3648 warps and items of 16 pages and 16 rows, rotate_kernel 608 CTAs that look up 128 rows at a time."""
import numpy as np
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests import select_ref
from tests.test_gpu_kv4_cache import ints
from tests.test_gpu_kv4_rotate import Rotated
from tests.test_gpu_kv4_select import Case as Selected
from tests.test_gpu_tokens import Case as Logits

pytestmark = pytest.mark.gpu


def some_slots(n):
    """Slots in another order than the requests, with requests of none in between."""
    return [-1 if i % 7 == 3 else n if i % 50 == 0 else int(s) for i, s in enumerate(np.random.default_rng(n).permutation(n))]


LOGITS = [
    dict(batch=1300, drafts=0, vocab=2104, dtype="bf16", out="f32", mask="picked"),
    dict(batch=1300, drafts=2, vocab=2104, dtype="f32", out="f32"),
    dict(batch=1300, drafts=2, vocab=2104, dtype="bf16", out="bf16", mask="picked", slots=some_slots(1300)),
    dict(batch=1300, drafts=2, vocab=2101, dtype="bf16", out="f32", slots=some_slots(1300)),
    dict(batch=1300, drafts=0, vocab=2101, dtype="f32", out="f32", mask="picked"),
    dict(batch=1300, drafts=2, vocab=2101, dtype="bf16", out="bf16", mask=None),
    dict(batch=800, drafts=9, vocab=2600, dtype="bf16", out="bf16"),  # more rows than masks come with a unit
    dict(batch=800, drafts=9, vocab=2600, dtype="f32", out="f32", mask="picked", slots=some_slots(800)),
    dict(batch=350, drafts=34, vocab=5120, dtype="bf16", out="f32", mask="picked"),  # more rows than a warp's lanes
    dict(batch=350, drafts=34, vocab=5117, dtype="bf16", out="bf16"),
    dict(batch=1100, drafts=1, vocab=2104, dtype="f32", out="f32", bias=60),  # more biases than stay in registers
    dict(batch=1100, drafts=1, vocab=2101, dtype="bf16", out="bf16", bias=60, slots=some_slots(1100), table=False),
]


@pytest.mark.parametrize("kw", LOGITS)
def test_adjusted_logits_of_several_units_a_warp(kw):
    c = Logits(**kw)
    assert -(-kw["vocab"] // 512) * kw["batch"] > 3040
    c.check()
    if kw["dtype"] == kw["out"]:
        want, x = c.run(), c.logits.clone()
        c.run(logits=x, out=x)
        assert torch.equal(x, want)


def check_selection(rows, lens, heads):
    """Random bounds: what a page's own would be is tested elsewhere."""
    rng = np.random.default_rng(4)
    c = Selected(rows=rows, lens=lens, page=16, heads=heads, group=2, dim=64, top=24, first=1, last=2, normal=False)
    c.ref_bounds[:] = rng.integers(0, 256, c.ref_bounds.shape, dtype=np.uint8)
    m = np.exp(rng.standard_normal((c.ref.num_pages, heads))).astype(np.float32)
    records = c.ref_bounds.reshape(c.ref.num_pages, heads, -1)
    records[:, :, 128:132] = m[..., None].view(np.uint8)
    c.bounds.copy_(torch.from_numpy(c.ref_bounds))
    pages, kept = c.select()
    q = c.q.float().cpu().numpy()
    for i in range(len(rows)):
        for j in range(rows[i]):
            row, pos = c.start[i] + j, lens[i] - rows[i] + j
            assert kept[row] == 23 * 16 + pos % 16 + 1
            for h in range(heads):
                ids = c.table[i][:pos // 16 + 1]
                rec = records[ids, h]  # all pages at once, as select_ref.select has them one by one
                a, b = select_ref.parts_of(q[row, 2 * h:2 * h + 2], False)
                lo, hi = (rec[:, w * 64:(w + 1) * 64].view(np.int8).astype(np.int64) for w in (0, 1))
                score = rec[:, 128:132].copy().view(np.float32)[:, 0] * (lo @ a + hi @ b).astype(np.float32)
                score[:1], score[-2:] = np.inf, np.inf
                want = ids[np.sort(np.argsort(-score, kind="stable")[:24])]
                assert np.array_equal(pages[row, h], want), (row, h)


@pytest.mark.parametrize("rows", [[1] * 16, [1, 0, 17, 3, 1, 33, 1, 2, 1, 16, 1, 5, 1, 0, 1, 1]])
def test_selections_of_several_items_a_warp(rows):
    lens = [16 * 700 + 5, 16 * 650] + [int(n) for n in np.random.default_rng(5).integers(16 * 500, 16 * 700, 14)]
    assert sum(-(-r // 16) * -(-n // 256) for r, n in zip(rows, lens)) * 8 > 4000
    check_selection(rows, lens, 8)


@pytest.mark.parametrize("most,requests,heads,rows", [
    (1024, 128, 4, 1), (1025, 128, 4, 1), (1024, 127, 4, 1), (512, 64, 4, 1), (513, 64, 4, 1),  # rows of one request each
    (320, 50, 4, 1), (321, 50, 4, 1), (128, 400, 2, 1), (129, 400, 2, 1),
    (576, 20, 5, 3), (577, 20, 5, 3), (320, 60, 4, 2), (321, 60, 4, 2), (129, 3, 2, 40),        # of several
    (2048, 20, 4, 1), (2049, 20, 4, 1), (300, 20, 4, 1), (300, 27, 3, 1), (256, 8, 4, 1), (256, 11, 3, 1)])  # few lists
def test_selections_on_both_sides_of_what_chooses_their_launches(most, requests, heads, rows):
    rng = np.random.default_rng(most)
    lens = [16 * most, 16 * most - 3] + [int(n) for n in rng.integers(16 * 30, 16 * most, requests - 2)]
    check_selection([rows] * requests, lens, heads)


@pytest.mark.parametrize("q_heads,dims", [(2, 64), (1, 32)])
def test_a_rotated_append_of_several_windows_a_cta(q_heads, dims):
    """Against the same rows in calls of few rows a CTA, which are tested against the formula."""
    rows = [31003, 50021, 7]
    kw = dict(rows=rows, lens=[31003, 60000, 7], page=256, heads=1, dim=64, q_heads=q_heads, dims=dims, positions=60000)
    c, d = Rotated(**kw), Rotated(**kw)
    assert c.total > 608 * 128
    got, want = torch.full_like(c.q, 9.0), torch.full_like(c.q, 9.0)
    binding.dspark_kv4_append_rotated(c.cache, c.batch, c.rotation, c.k, c.v, c.q, got)
    for i, n in enumerate(rows):
        for first in range(0, n, 20000):
            last = min(first + 20000, n)
            here = slice(c.start[i] + first, c.start[i] + last)
            held = c.slot_lens.copy()
            held[i] -= n - last
            batch = binding.Kv4Batch(ints([0, last - first]), ints(held), ints(c.table), total_rows=last - first,
                                     max_rows=last - first, slots=ints([i]))
            binding.dspark_kv4_append_rotated(d.cache, batch, d.rotation, d.k[here], d.v[here], d.q[here], want[here])
    assert torch.equal(c.data, d.data)
    assert torch.equal(got, want) and not (got == 9.0).all(2).any()
