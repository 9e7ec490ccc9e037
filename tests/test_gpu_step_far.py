"""Lists at the end of what 31 bits count: arguments as large as the headers allow, of which few are used."""
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests.test_gpu_kv4_cache import ints

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()  # what these take is given back


def test_a_selection_of_as_many_pages_as_there_are_numbers():
    page, heads, dim, n = 16, 1, 64, 100
    cache = binding.Kv4Cache(torch.zeros(8, binding.kv4_page_bytes(page, heads, dim), dtype=torch.uint8, device="cuda"),
                             page, heads, dim)
    batch = binding.Kv4Batch(ints([0, 1]), ints([n]), ints([[3, 1, 0, 2, 7, 6, 5]]), total_rows=1, max_rows=1)
    pages = torch.full((1, heads, MOST), -77, dtype=torch.int32, device="cuda")
    lens = ints([-77])
    selection = binding.Kv4Selection(pages, lens)
    bounds = torch.zeros(8, binding.kv4_bounds_bytes(heads, dim), dtype=torch.uint8, device="cuda")
    work = torch.zeros(binding.dspark_kv4_select_workspace_bytes(cache, batch, selection), dtype=torch.uint8, device="cuda")
    q = torch.zeros(1, 1, dim, dtype=torch.bfloat16, device="cuda")
    binding.dspark_kv4_select(cache, batch, bounds, q, selection, work)
    assert lens.tolist() == [n] and pages[0, 0, :7].tolist() == [3, 1, 0, 2, 7, 6, 5]
    for part in pages[0, 0, 7:].split(1 << 28):
        assert (part == -1).all()


@pytest.mark.parametrize("reset", [False, True])
def test_as_many_lists_of_tokens_as_there_are_numbers(reset):
    """Slot i has list i, so that all but the first three are skipped unread."""
    counts = torch.full((3, 40), 5, dtype=torch.int32, device="cuda")
    marks = torch.zeros(3, 2, 2, dtype=torch.int32, device="cuda")
    tokens = torch.empty(MOST, 1, dtype=torch.int32, device="cuda")
    lens = torch.empty(MOST, dtype=torch.int32, device="cuda")
    tokens[:3, 0], lens[:3] = ints([7, 39, 33]), ints([1, 0, 1])
    binding.dspark_tokens_count(binding.TokenTable(counts, marks), tokens, lens, reset=reset)
    want = torch.full((3, 40), 0 if reset else 5, dtype=torch.int32)
    want[0, 7] += 1
    want[2, 33] += 1
    assert torch.equal(counts.cpu(), want)
    assert marks.flatten(1).tolist() == [[0, 0, 1 << 7, 0], [0, 0, 0, 0], [0, 0, 0, 2]]


@pytest.mark.parametrize("n", [1, 40, 65, 100])
def test_the_last_of_as_many_biases_as_there_are_numbers(n):
    ids, values = (torch.empty(MOST, dtype=t, device="cuda") for t in (torch.int32, torch.float32))
    ids[-n:] = torch.arange(n, device="cuda") * 7
    values[-n:] = torch.arange(1, n + 1, device="cuda") / 4
    x = torch.zeros(2, 5000, device="cuda")
    binding.dspark_logits_adjust(None, x, x, bias=(ints([MOST - n, MOST, MOST]), ids, values))
    want = torch.zeros(2, 5000)
    want[0, torch.arange(n) * 7] = torch.arange(1, n + 1) / 4
    assert torch.equal(x.cpu(), want)


def test_as_many_rows_as_there_are_numbers():
    """Rows that share one key and value; all but the last 16 are before their request's first token."""
    size, n = binding.kv4_page_bytes(16, 1, 64), 16
    angle = torch.arange(n, device="cuda")[:, None] * torch.linspace(1.0, 0.01, 32, device="cuda")
    rotation = binding.Kv4Rotation(angle.cos(), angle.sin())
    k, v = (torch.linspace(a, b, 64, device="cuda").to(torch.bfloat16).view(1, 1, 64) for a, b in ((-3, 2), (1, 5)))
    data = torch.zeros(2, 3, size, dtype=torch.uint8, device="cuda")
    for x, rows in zip(data, (MOST, n)):
        cache = binding.Kv4Cache(x, 16, 1, 64)
        batch = binding.Kv4Batch(ints([0, rows]), ints([n]), ints([[2]]), total_rows=rows, max_rows=rows)
        binding.dspark_kv4_append_rotated(cache, batch, rotation, k.expand(rows, 1, 64), v.expand(rows, 1, 64))
    assert torch.equal(data[0], data[1]) and data[0, 2].any() and not data[0, :2].any()
