"""Attention calls whose units (tiles of rows, with a head) and blocks of 64 tokens number more than 32 bits hold.  One
that promises few rows and has many gets larger tiles: compared with the same call made with the rows that it has, which
tests/test_gpu_kv4_attention.py compares with 64 bits.  One too long for any tile is NaN."""
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests.test_gpu_kv4_cache import ints

pytestmark = pytest.mark.gpu


def test_more_rows_than_promised_in_a_long_call():
    requests, rows, heads, group, dim, page = 8, 1 << 16, 8, 8, 64, 64
    total, pages = requests * rows, rows // page
    tiles = total * group // 8
    assert heads * tiles * (rows // 64 // 2 + 5) > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(1)
    start = ints([i * rows for i in range(requests + 1)])
    lens = ints([rows] * requests)
    table = torch.randperm(requests * pages, device="cuda", generator=gen).int().view(requests, pages)
    data = torch.zeros(requests * pages, binding.kv4_page_bytes(page, heads, dim), dtype=torch.uint8, device="cuda")
    cache = binding.Kv4Cache(data, page, heads, dim)
    k, v = (torch.randn(total, heads, dim, dtype=torch.bfloat16, device="cuda", generator=gen) for _ in range(2))
    batches = [binding.Kv4Batch(start, lens, table, total_rows=total, max_rows=n) for n in (1, rows)]
    binding.dspark_kv4_append(cache, batches[0], k, v)
    binding.dspark_kv4_read(cache, batches[0], None, v)
    most = v.abs().max().item()
    del k, v
    q = torch.randn(total, heads * group, dim, dtype=torch.bfloat16, device="cuda", generator=gen)
    got = []
    for batch in batches:
        out, lse = torch.full_like(q, -55.0), torch.full(q.shape[:2], -55.0, device="cuda")
        work = torch.empty(binding.dspark_kv4_attention_workspace_bytes(cache, batch, heads * group), dtype=torch.uint8,
                           device="cuda")
        binding.dspark_kv4_attention(cache, batch, q, out, dim ** -0.5, work, lse=lse)
        got.append((out, lse))
    torch.cuda.synchronize()
    (a, la), (b, lb) = got
    # each is within (2^-11 + 2 d) sum p |v| / sum p and its own rounding, 2^-9, of the exact value, the logarithms
    # within d; sum p |v| / sum p is at most the largest value, and d, for scores of a dot product below 2^6, 2^-11
    assert (la - lb).abs().max() < 2.0 ** -9
    for i in range(requests):
        x, y = a[i * rows:(i + 1) * rows].float(), b[i * rows:(i + 1) * rows].float()
        assert ((x - y).abs() <= 2 * 3 * 2.0 ** -11 * most + 2.0 ** -7 * y.abs()).all(), i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_rows", [1, 100, 10000])
def test_a_call_that_is_too_long(dim, dtype, max_rows):
    """4000 requests of one row and 64 heads over 2^20 tokens: 4.2e9 blocks.  Their pages are not there (and not
    read)."""
    n, heads, page = 4000, 64, 256
    table = ints([[-1] * ((1 << 20) // page)])
    cache = binding.Kv4Cache(torch.zeros(1, binding.kv4_page_bytes(page, heads, dim), dtype=torch.uint8, device="cuda"),
                             page, heads, dim)
    q = torch.randn(n + 2, heads, dim, device="cuda").to(dtype)

    def run(length, n):
        batch = binding.Kv4Batch(ints(range(1, n + 2)), ints([length]), table, total_rows=n + 2, max_rows=max_rows,
                                 slots=ints([0] * n))
        out, lse = torch.full_like(q, -55.0), torch.full(q.shape[:2], -55.0, device="cuda")
        work = torch.empty(binding.dspark_kv4_attention_workspace_bytes(cache, batch, heads), dtype=torch.uint8,
                           device="cuda")
        binding.dspark_kv4_attention(cache, batch, q, out, 1.0, work, lse=lse)
        return out, lse
    out, lse = run(1 << 20, n)
    assert torch.isnan(out[1:-1]).all() and torch.isnan(lse[1:-1]).all()
    assert (out[0] == -55).all() and (out[-1] == -55).all() and (lse[0] == -55).all() and (lse[-1] == -55).all()
    # the same tables and shorter requests: computed (nothing is seen)
    out, lse = run(300, n)
    assert (out[1:-1] == 0).all() and torch.isneginf(lse[1:-1]).all()
