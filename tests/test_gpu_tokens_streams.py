"""Token counts and adjusted logits on a stream that is not the current one: what they read comes late on that stream,
so that a call on any other one would not see it."""
import numpy as np
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests.test_gpu_kv4_cache import ints
from tests.test_gpu_tokens import Case, Table

pytestmark = pytest.mark.gpu


def late(*pairs):
    """A stream on which each tensor gets its values after a while."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        for to, values in pairs:
            to.copy_(values)
    return s


@pytest.mark.parametrize("kinds", [("bf16", "f32"), ("bf16", "bf16")])
def test_adjusted_logits(kinds):
    c = Case(3, 2, 4000, dtype=kinds[0], out=kinds[1])
    want, a = c.run(), c.arguments()
    logits, draft = c.logits.clone(), a["draft"].clone()
    out = torch.empty_like(want)
    c.logits.zero_()
    a["draft"].fill_(-1)
    s = late((c.logits, logits), (a["draft"], draft))
    binding.dspark_logits_adjust(c.t.table, c.logits, out, stream=s, **a)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    if kinds[0] == kinds[1]:
        c.logits.zero_()
        s = late((c.logits, logits))
        binding.dspark_logits_adjust(c.t.table, c.logits, c.logits, stream=s, **a)
        torch.cuda.synchronize()
        assert torch.equal(c.logits, want)


@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("n,width", [(5, 300), (40, 20000)])  # the second marks in shared memory
def test_token_counts(n, width, reset, prompt):
    rng = np.random.default_rng(width)
    t = Table(n, 5000)
    tokens, lens, slots = rng.integers(0, 5000, (n, width)), rng.integers(0, width + 1, n), rng.permutation(n)
    ids, held, at = torch.from_numpy(tokens).cuda(), ints(lens), ints(slots)
    late_ids, late_held, late_at = torch.zeros_like(ids), torch.zeros_like(held), torch.zeros_like(at)
    before = torch.full_like(t.counts, 3)
    s = late((late_ids, ids), (late_held, held), (late_at, at), (t.counts, before))
    binding.dspark_tokens_count(t.table, late_ids, late_held, slots=late_at, prompt=prompt, reset=reset, stream=s)
    torch.cuda.synchronize()
    want = np.zeros((n, 5000), np.int64)
    for i in range(n):
        want[slots[i]] = np.bincount(tokens[i][:lens[i]], minlength=5000)
    if prompt:
        t.prompt, t.want = want > 0, np.zeros_like(want) if reset else np.full_like(want, 3)
        assert np.array_equal(t.counts.cpu().numpy(), t.want)
        t.want[:] = 0  # the marks of outputs are of what was counted, which nothing was
        t.counts.zero_()
    else:
        if not reset:
            assert np.array_equal(t.counts.cpu().numpy(), want + 3)
            t.counts -= 3
        t.want = want
    t.check()
