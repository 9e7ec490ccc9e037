"""Pages and bounds that begin more than 2^32 bytes behind the first: the last pages of a large pool, and of a small one,
hold the same bytes and give the same results."""
import numpy as np
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests import kv4_ref
from tests.test_gpu_kv4_cache import ints

pytestmark = pytest.mark.gpu
PAGE, HEADS, DIM = 64, 2, 128
SIZE = binding.kv4_page_bytes(PAGE, HEADS, DIM)


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()  # what these take is given back


class Pool:
    """Pages `apart` bytes from one another, with others' bytes around them."""

    def __init__(self, num_pages, size, apart):
        self.all = torch.zeros(num_pages, apart, dtype=torch.uint8, device="cuda")
        self.here = self.all[:, 16:16 + size]

    def untouched(self, but):
        assert not self.all[:, :16].any() and not self.all[:, 16 + self.here.shape[1]:].any()
        return not self.all[:len(self.all) - but].any()


@pytest.mark.parametrize("seed", range(3))
def test_rows_stored_and_read(seed):
    rng = np.random.default_rng(seed)
    pool = Pool((1 << 32) // (3 * SIZE) + 10, SIZE, 3 * SIZE)
    last = len(pool.all) - 1
    cache = binding.Kv4Cache(pool.here, PAGE, HEADS, DIM)
    batch = binding.Kv4Batch(ints([0, PAGE]), ints([PAGE]), ints([[last]]), total_rows=PAGE, max_rows=PAGE)
    x = torch.from_numpy(rng.standard_normal((2, PAGE, HEADS, DIM))).to(torch.bfloat16)
    binding.dspark_kv4_append(cache, batch, x[0].cuda(), x[1].cuda())
    got = torch.empty(2, PAGE, HEADS, DIM, dtype=torch.bfloat16, device="cuda")
    binding.dspark_kv4_read(cache, batch, got[0], got[1])
    x = x.double().numpy()
    code, scale = kv4_ref.quantise(x, 1.0)
    assert torch.equal(got.cpu(), torch.from_numpy(kv4_ref.values(code, scale, 1.0)).to(torch.bfloat16))
    # The scale is a sixth of its 16 elements' largest, M, off by at most 2^-4 of itself.  Up to 6 scales the gap
    # between codes is at most 2 scales, so that an element is off by at most one; what is above 6 scales is off by at
    # most 2^-4 M, which is less.  Then half a step of BF16.
    most = np.abs(x).reshape(2, PAGE, HEADS, -1, 16).max(-1).repeat(16, -1) / 6 * (1 + 2.0 ** -4) * (1 + 2.0 ** -20)
    off = np.abs(got.double().cpu().numpy() - x)
    assert np.all(off <= most + 2.0 ** -8 * (np.abs(x) + most))
    assert pool.untouched(but=1)


def test_a_step_over_a_long_context():
    """Rotated rows, bounds, selection and attention over the selection."""
    n, q_heads, top = 9 * PAGE + 17, 4, 5
    rng = np.random.default_rng(7)
    x = [torch.from_numpy(rng.standard_normal((n, h, DIM))).to(torch.bfloat16).cuda() for h in (HEADS, HEADS, q_heads)]
    angle = torch.arange(n, device="cuda")[:, None] * torch.linspace(1.0, 0.001, DIM // 2, device="cuda")
    rotation = binding.Kv4Rotation(angle.cos(), angle.sin())
    size = binding.kv4_bounds_bytes(HEADS, DIM)
    results = []
    many = (1 << 32) // (2 * SIZE) + 20
    for num_pages, apart, bounds_apart in ((12, SIZE + 64, size + 32), (many, 2 * SIZE, ((1 << 32) // many + 256) // 16 * 16)):
        data, bounds = Pool(num_pages, SIZE, apart), Pool(num_pages, size, bounds_apart)
        cache = binding.Kv4Cache(data.here, PAGE, HEADS, DIM)
        table = ints([[num_pages - 1 - p for p in rng.permutation(10)] if not results else
                      [num_pages - 12 + int(p) for p in results[0][0]]])
        batch = binding.Kv4Batch(ints([0, n]), ints([n]), table, total_rows=n, max_rows=n)
        q, out = torch.empty_like(x[2]), torch.empty_like(x[2])
        binding.dspark_kv4_append_rotated(cache, batch, rotation, x[0], x[1], x[2], q)
        binding.dspark_kv4_bound_pages(cache, batch, bounds.here)
        pages, lens = torch.empty(n, HEADS, top, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
        chosen = binding.Kv4Selection(pages, lens)
        work = torch.zeros(max(binding.dspark_kv4_select_workspace_bytes(cache, batch, chosen),
                               binding.dspark_kv4_attention_selected_workspace_bytes(cache, chosen, q_heads)),
                           dtype=torch.uint8, device="cuda")
        binding.dspark_kv4_select(cache, batch, bounds.here, q, chosen, work)
        binding.dspark_kv4_attention_selected(cache, chosen, q, out, DIM ** -0.5, work)
        few = binding.Kv4Batch(ints([0, 3]), ints([n]), table, total_rows=3, max_rows=3)  # bounds of few rows
        first = bounds.here[-12:].clone()
        binding.dspark_kv4_bound_pages(cache, few, bounds.here)
        assert torch.equal(first, bounds.here[-12:]) and first.any()
        base = num_pages - 12
        results.append((table[0] - base, q, data.here[-12:].clone(), first, torch.where(pages < 0, pages, pages - base),
                        lens, out))
        assert data.untouched(but=12) and bounds.untouched(but=12)
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert data.all.numel() > 1 << 32 and bounds.all.numel() > 1 << 32
