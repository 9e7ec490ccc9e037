"""Numbers of heads behind which places of a line of heads, or the queries of a group, would not be counted in 31 bits
are refused before any CUDA call (no GPU needed)."""
import pytest

from tests.test_kv4_arguments import INVALID, batch, cache
from tests.test_step_arguments import lib, rotated, select  # noqa: F401


@pytest.mark.parametrize("q_heads", [2 ** 31 - 5, 2 ** 31 - 1024 - 4, 2 ** 31 - 1])
def test_query_heads_of_a_rotated_append(lib, q_heads):  # noqa: F811
    assert rotated(lib, args=dict(q_heads=q_heads, q_head=0)) == INVALID
    assert rotated(lib, c=cache(), b=batch(total_rows=0), args=dict(q_heads=2 ** 31 - 1025 - 4)) == 0


@pytest.mark.parametrize("q_heads", [2 ** 30 + 1, 2 ** 31 - 2, 2 ** 31 - 1])
def test_queries_of_a_selections_group(lib, q_heads):  # noqa: F811
    c, one = cache(kv_heads=1), dict(rows=1)
    assert select(lib, c, batch(total_rows=1), selection=one, args=dict(q_heads=q_heads, q_head=0)) == INVALID
