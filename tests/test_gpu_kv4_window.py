"""Attention over the paged 4-bit cache with windows up to the type's largest number, also where requests have more
rows than tokens: such a window is none."""
import pytest
import torch

from tests.test_gpu_kv4_attention import Case

pytestmark = pytest.mark.gpu
LARGE = 2 ** 31 - 1


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kw", [
    dict(rows=[6], lens=[2], page=16, heads=1, group=1, dim=64),
    dict(rows=[6, 40, 3], lens=[2, 30, 90], page=32, heads=1, group=8, dim=128),
    dict(rows=[150, 7], lens=[70, 0], page=64, heads=2, group=2, dim=64, dtype="f16"),
    dict(rows=[70], lens=[5], page=64, heads=1, group=8, dim=128),
])
def test_a_window_as_large_as_the_type(kw, wide):
    want, want_lse = Case(wide=wide, **kw).run()
    for window in (LARGE, LARGE - 1, LARGE - 70, 1 << 30, 30000 * kw["page"]):
        c = Case(wide=wide, window=window, **kw)
        out, lse = c.run()
        assert torch.equal(out, want) and torch.equal(lse, want_lse), window
    c.check()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("window", [1, 3, 64, 65])
def test_a_window_and_rows_at_negative_positions(window, wide):
    Case([90, 20, 300], [66, 3, 129], 32, 1, 2, 64, window=window, wide=wide).check()
