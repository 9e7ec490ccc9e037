"""Scores as large as include/dspark_kv4.h allows, 2^23 in magnitude: rows are weighted like any other."""
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests.test_gpu_kv4_attention import Case
from tests.test_gpu_kv4_cache import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("rows,dim,dtype", [(1, 64, "bf16"), (5, 128, "f16"), (20, 128, "bf16"), (40, 64, "f16")])
def test_scores_far_from_zero(rows, dim, dtype, wide):
    """One token, or equal ones: their weights are equal whatever the scores are, so the result is their value."""
    for most in (2.0 ** 10, 2.0 ** 17, 2.0 ** 23):
        for sign in (1, -1):
            c = Case([rows], [rows], 16, 1, 8, dim, dtype=dtype, wide=wide, seed=rows)
            k, v = (torch.empty(1, 1, dim, device="cuda") for _ in range(2))
            x = torch.randn(1, 1, dim, device="cuda").to(c.q.dtype).expand(rows, 1, dim)
            binding.dspark_kv4_append(c.cache, c.batch, x, x)
            one = binding.Kv4Batch(ints([0, 1]), ints([1]), ints(c.table[:1]), total_rows=1, max_rows=1)
            binding.dspark_kv4_read(c.cache, one, k, v)
            dots = c.q.double() @ k[0, 0].double()
            c.scale = sign * most / dots.abs().max().item()
            out, lse = c.run()
            # weights that are alike leave the value but for the sums' and the result's rounding
            unit = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
            assert ((out.float() - v).abs() <= (unit + 1e-5) * v.abs()).all(), most
            # the dot product's terms are off by 2^-24 each and there are dim of them; the logarithm of up to 40 weights
            size = c.q.double().abs() @ k[0, 0].double().abs() * abs(c.scale)
            tokens = torch.arange(1, rows + 1, device="cuda", dtype=torch.float64)[:, None]
            want = dots * c.scale + torch.log(tokens)
            assert ((lse.double() - want).abs() <= (dim + 8) * 2.0 ** -24 * size + 1e-5).all(), most
