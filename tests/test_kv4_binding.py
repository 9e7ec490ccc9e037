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
