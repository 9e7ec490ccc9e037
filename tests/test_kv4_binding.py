"""The binding of the paged 4-bit cache refuses tensors that the kernels would read or write otherwise than they are
laid out.  Everything here is refused before the library is called (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

from dspark_markov_draft_anchor_gb300 import binding  # noqa: E402


def step(rows=3, heads=2, dim=64):
    cache = binding.Kv4Cache(torch.zeros(4, binding.kv4_page_bytes(16, heads, dim), dtype=torch.uint8), 16, heads, dim)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    batch = binding.Kv4Batch(ints(0, rows), ints(rows), torch.zeros(1, 4, dtype=torch.int32), total_rows=rows,
                             max_rows=rows)
    return cache, batch


@pytest.mark.parametrize("lse", [torch.zeros(3, 4, dtype=torch.bfloat16), torch.zeros(3, 4, dtype=torch.float16),
                                 torch.zeros(3, 4, dtype=torch.float64), torch.zeros(3, 4, dtype=torch.int32),
                                 torch.zeros(12), torch.zeros(3, 4, 1), torch.zeros(2, 4), torch.zeros(3, 5),
                                 torch.zeros(4, 3).T])
def test_lse_is_float32_rows_by_heads(lse):
    cache, batch = step()
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises((ValueError, TypeError)):
        binding.dspark_kv4_attention(cache, batch, q, torch.empty_like(q), 0.1, torch.empty(0, dtype=torch.uint8),
                                     lse=lse)


ROWS = torch.zeros(6, 8, dtype=torch.int32)
LISTS = [ROWS[:, :1], ROWS[:, 0], ROWS[::2], ROWS[:, :4], torch.zeros(1, dtype=torch.int32).expand(6),
         torch.zeros(6, dtype=torch.int64)]


@pytest.mark.parametrize("bad", LISTS)
def test_lists_are_contiguous(bad):
    good = torch.zeros(bad.numel(), dtype=torch.int32)
    table = torch.zeros(bad.numel(), 4, dtype=torch.int32)
    for kw in (dict(row_start=bad, lens=good), dict(row_start=good, lens=bad)):
        with pytest.raises((TypeError, ValueError)):
            binding.Kv4Batch(kw["row_start"], kw["lens"], table, total_rows=1, max_rows=1)
    with pytest.raises((TypeError, ValueError)):
        binding.Kv4Batch(torch.zeros(bad.numel() + 1, dtype=torch.int32), good, table, total_rows=1, max_rows=1, slots=bad)
    for refs, lens in ((bad, good), (good, bad)):
        with pytest.raises((TypeError, ValueError)):
            binding.PagePool(refs, table, lens, 16)


@pytest.mark.parametrize("bad", [torch.zeros(6, dtype=torch.int32), ROWS.T[:6, :4], ROWS[:, ::2],
                                 torch.zeros(6, 2, 2, dtype=torch.int32), torch.zeros(6, 8)])
def test_tables_are_rows_of_pages(bad):
    good = torch.zeros(6, dtype=torch.int32)
    with pytest.raises((TypeError, ValueError)):
        binding.Kv4Batch(good, good, bad, total_rows=1, max_rows=1)
    with pytest.raises((TypeError, ValueError)):
        binding.PagePool(good, bad, good, 16)


def test_tables_may_be_part_of_wider_ones():
    good = torch.zeros(6, dtype=torch.int32)
    for table in (ROWS, ROWS[:, :4], ROWS[:, :1], ROWS[::2]):
        lens = good[:table.shape[0]]
        assert binding.Kv4Batch(good, lens, table, total_rows=1, max_rows=1).struct.table_stride == table.stride(0)
        assert binding.PagePool(good, table, lens, 16).struct.max_pages == table.shape[1]
