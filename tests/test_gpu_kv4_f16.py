"""FP16 results are as near to the 64-bit values whichever kernel a call takes.

Weights enter the second product as two FP16 numbers, 21 bits: off by a share of 2^-21, or 2^-25 where the second is
one of FP16's smallest numbers, which is 2^-30 of the row's largest weight (weights are 2^5 there).  With the score's
share d of tests/kv4_ref.py that leaves (2^-21 + 2 d) sum p |v| + 2^-29 sum |v|, and the result's own rounding,
2^-11.  One FP16 number would add 2^-11 sum p |v|, which small scores (d of 2^-20) and values that cancel show."""
import pytest
import torch

from tests.test_gpu_kv4_attention import Case, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kw", [
    dict(rows=[1, 2], lens=[300, 70], page=64, heads=2, group=4, dim=128),
    dict(rows=[6, 6], lens=[1000, 64], page=64, heads=2, group=8, dim=128),
    dict(rows=[40, 1, 9], lens=[700, 65, 2000], page=16, heads=1, group=5, dim=64, window=500),
    dict(rows=[200, 33], lens=[900, 4000], page=32, heads=1, group=4, dim=128),
    dict(rows=[257, 3], lens=[600, 300], page=128, heads=2, group=2, dim=64),
])
def test_fp16_results(kw, wide):
    c = Case(dtype="f16", scale=1e-3, seed=11, wide=wide, **kw)
    out, _ = c.run()
    want, tol, size = on_gpu(c) + (on_gpu_size(c),)
    room = 1.01 * (tol - (2.0 ** -11 - 2.0 ** -21) * size) + 2.0 ** -11 * want.abs() + 2.0 ** -24
    err = (out.double() - want).abs()
    assert (err <= room).all(), (err / room).max()


def on_gpu_size(c):
    """sum p |v| of each output: the values' magnitudes under the same weights."""
    import copy
    m = copy.copy(c)
    m.data = c.data.clone()
    half, eighth = c.ref.page * c.dim // 2, c.ref.page * c.dim // 16
    r = m.data.view(c.ref.num_pages, c.heads, -1)
    r[:, :, half:2 * half] &= 0x77
    r[:, :, 2 * half + eighth:2 * (half + eighth)] &= 0x7F
    from dspark_markov_draft_anchor_gb300 import binding
    m.cache = binding.Kv4Cache(m.data, c.ref.page, c.heads, c.dim)
    return on_gpu(m)[0]
