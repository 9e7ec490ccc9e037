"""Storing rows with rotated keys: the formula in FP32, operation by operation (numpy rounds each as the kernel has
to), gives the same bytes of the cache and the same rotated queries, bit for bit."""
import numpy as np
import pytest
import torch

from dspark_markov_draft_anchor_gb300 import binding
from tests import kv4_ref
from tests.test_gpu_kv4_cache import TYPES, Case, ints

pytestmark = pytest.mark.gpu
F = np.float32


def quantise32(x, g):
    """FP32 x [..., 16 n] -> codes and scales, by FP32 quotients."""
    with np.errstate(all="ignore"):
        y = (x / F(g)).astype(F)
        y = np.where(np.isnan(y), F(0), y).reshape(*x.shape[:-1], -1, 16)
        top = (np.abs(y).max(-1) / F(6)).astype(F)
        scale = kv4_ref.nearest(kv4_ref.POSITIVE, np.minimum(top, F(448)).astype(np.float64)).astype(np.uint8)
        s = kv4_ref.POSITIVE[scale].astype(F)[..., None]
        a = np.where(s > 0, np.minimum((np.abs(y) / s).astype(F), F(6)), F(0))
    code = kv4_ref.nearest(kv4_ref.E2M1, a.astype(np.float64)) + 8 * (y < 0)
    return code.astype(np.uint8).reshape(x.shape), scale


def rotate32(x, cos, sin, interleaved):
    """FP32 x [heads, dim], cos and sin [dims / 2]."""
    out, n = x.copy(), 2 * len(cos)
    first = slice(0, n, 2) if interleaved else slice(0, n // 2)
    second = slice(1, n, 2) if interleaved else slice(n // 2, n)
    with np.errstate(all="ignore"):
        a, b = x[:, first], x[:, second]
        out[:, first] = a * cos - b * sin
        out[:, second] = b * cos + a * sin
    return out


class Rotated(Case):
    def __init__(self, rows, lens, page, heads, dim, *, q_heads=4, dims=None, interleaved=False, given=None, positions=600,
                 q_seed=5, **kw):
        super().__init__(rows, lens, page, heads, dim, **kw)
        rng = np.random.default_rng(q_seed)
        self.q = torch.from_numpy(rng.standard_normal((self.total, q_heads, dim))).to(self.k.dtype).cuda()
        self.dims, self.interleaved = dims or dim, interleaved
        angle = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(self.dims // 2) / (self.dims // 2))
        self.cos, self.sin = np.cos(angle).astype(F), np.sin(angle).astype(F)
        self.given = given
        self.rotation = binding.Kv4Rotation(torch.from_numpy(self.cos).cuda(), torch.from_numpy(self.sin).cuda(),
                                            interleaved=interleaved, positions=None if given is None else ints(given))

    def wants(self):
        """Stores what the call has to store; returns the rotated queries as FP32, NaN for rows that have none."""
        q = np.full(self.q.shape, np.nan, F)
        k, v, qs = (t.float().cpu().numpy() for t in (self.k, self.v, self.q))
        wide = np.zeros(self.total, bool)  # rows of a request
        for i, s in enumerate(self.slots):
            for j in range(self.rows[i]):
                row, pos = self.start[i] + j, self.slot_lens[s] - self.rows[i] + j
                wide[row] = True
                if pos < 0:
                    q[row] = 0
                    continue
                at = pos if self.given is None else self.given[row]
                if not 0 <= at < len(self.cos):
                    continue
                c, sn = self.cos[at], self.sin[at]
                q[row] = rotate32(qs[row], c, sn, self.interleaved)
                p = self.table[s, pos // self.page]
                if not 0 <= p < self.ref.num_pages:
                    continue
                turned = rotate32(k[row], c, sn, self.interleaved)
                for h in range(self.heads):
                    codes, scales = self.ref.sections(p, h)
                    for w, x in enumerate((turned[h], v[row, h])):
                        c4, s8 = quantise32(x, self.ref.g[w][h])
                        codes[w][pos % self.page] = c4[0::2] | (c4[1::2] << 4)
                        scales[w][pos % self.page] = s8
        assert wide.all()
        return q

    def check(self, q=None, out=None):
        want = self.wants()
        q = self.q if q is None else q
        out = torch.empty_like(self.q) if out is None else out
        binding.dspark_kv4_append_rotated(self.cache, self.batch, self.rotation, self.k, self.v, q, out)
        torch.cuda.synchronize()
        same_bytes(self)
        got = out.float().cpu().numpy()
        wanted = torch.from_numpy(want).to(self.q.dtype).float().numpy()
        assert np.array_equal(got, wanted, equal_nan=True)


def same_bytes(c):
    """The cache's bytes; a code's sign where the magnitude is 0 is free."""
    got = c.data.cpu().numpy()
    for p, at in np.argwhere(got != c.ref.data):
        assert at % c.ref.record < c.page * c.dim, "a scale differs"
        a, b = int(got[p, at]), int(c.ref.data[p, at])
        for sh in (0, 4):
            x, y = a >> sh & 15, b >> sh & 15
            assert x == y or (x & 7) == (y & 7) == 0, (p, at, a, b)


CASES = [
    dict(rows=[1], lens=[1], page=16, heads=1, dim=64, q_heads=1),
    dict(rows=[6, 6, 6], lens=[100, 6, 71], page=64, heads=8, dim=128, q_heads=64),
    dict(rows=[6, 6, 6], lens=[100, 6, 71], page=64, heads=8, dim=128, q_heads=64, interleaved=True),
    dict(rows=[0, 1, 0, 33, 2], lens=[5, 17, 0, 33, 1], page=16, heads=5, dim=64, q_heads=7, dtype="f16", dims=32),
    dict(rows=[0, 1, 0, 33, 2], lens=[5, 17, 0, 33, 1], page=16, heads=5, dim=64, q_heads=7, dims=32, interleaved=True),
    dict(rows=[5, 7], lens=[3, 300], page=256, heads=2, dim=128, q_heads=2, gk=[0.25, 4.0], gv=[1.0, 2.0 ** -7], dims=96),
    dict(rows=[40], lens=[40], page=128, heads=3, dim=128, q_heads=5, spread=6.0, gk=[0.03, -1.7, 1e-9], gv=[3.3, 1e6, 0.2]),
    dict(rows=[129, 1], lens=[200, 257], page=32, heads=3, dim=128, slots=[4, 1], dtype="f16", q_heads=12, dims=64),
    dict(rows=[3, 2], lens=[20, 30], page=16, heads=2, dim=128, q_heads=16, given=[599, 0, 77, 600, -1]),
    dict(rows=[2, 1], lens=[20, 1], page=16, heads=2, dim=64, q_heads=3, positions=19),
    dict(rows=[1], lens=[40], page=16, heads=1, dim=64, q_heads=70),
    dict(rows=[1300], lens=[1300], page=64, heads=1, dim=64, q_heads=2, positions=1300),        # several rows a CTA
    dict(rows=[5000, 21], lens=[5000, 40], page=128, heads=1, dim=64, q_heads=1, positions=5000, dims=32),
]


@pytest.mark.parametrize("kw", CASES)
def test_bytes_and_queries(kw):
    Rotated(**kw).check()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinities_nan_and_the_largest_values(dtype, interleaved):
    c = Rotated(rows=[4], lens=[30], page=16, heads=3, dim=64, q_heads=3, dtype=dtype, interleaved=interleaved, dims=32)
    big = torch.finfo(TYPES[dtype]).max
    for t in (c.k, c.v, c.q):
        t[0, 0, 3], t[0, 1, 17], t[1, 0, 40] = float("inf"), float("nan"), float("-inf")
        t[1, 1, ::2], t[2, 0], t[3, 2, 5] = big, -big, big
    # the kernel's NaN is one pattern, numpy's any: compared as NaN
    c.check()


def test_strides_and_misaligned_rows():
    kw = dict(rows=[6, 9], lens=[50, 9], page=16, heads=2, dim=64, q_heads=6)
    for shift in (0, 1):
        c = Rotated(**kw)
        wide = torch.randn(c.total, 10 * 64 + 8 + shift, device="cuda").to(c.k.dtype)
        views = [wide[:, shift + a * 64:shift + b * 64].unflatten(1, (b - a, 64)) for a, b in ((0, 6), (6, 8), (8, 10))]
        for view, t in zip(views, (c.q, c.k, c.v)):
            view.copy_(t)
        c.k, c.v = views[1], views[2]
        c.check(q=views[0])
        c = Rotated(**kw)
        c.check(out=torch.empty(6, c.total, 64, dtype=c.q.dtype, device="cuda").transpose(0, 1))


def test_queries_in_place_and_keys_alone():
    c = Rotated(rows=[6, 9], lens=[50, 9], page=16, heads=2, dim=64, q_heads=6)
    q = c.q.clone()
    c.check(q=q, out=q)
    d = Rotated(rows=[6, 9], lens=[50, 9], page=16, heads=2, dim=64, q_heads=6)
    binding.dspark_kv4_append_rotated(d.cache, d.batch, d.rotation, d.k, d.v)
    assert torch.equal(c.data, d.data)


def test_table_rows_apart_and_unaligned():
    c = Rotated(rows=[6, 9], lens=[50, 9], page=16, heads=2, dim=64, q_heads=6)
    wide = torch.zeros(600, 2 * 32 + 3, device="cuda")
    wide[:, 1:33], wide[:, 34:66] = c.rotation.cos, c.rotation.sin
    c.rotation = binding.Kv4Rotation(wide[:, 1:33], wide[:, 34:66])
    c.check()


def test_rows_without_a_request_or_a_page_are_left():
    c = Rotated(rows=[3, 4], lens=[20, 9], page=16, heads=2, dim=64, q_heads=3)
    c.table[0, 1] = c.ref.num_pages + 3
    c.batch.tensors[2].copy_(ints(c.table))
    c.check()
    c = Rotated(rows=[3, 4], lens=[20, 9], page=16, heads=2, dim=64, q_heads=3)
    c.batch.tensors[0].copy_(ints([2, 3, 5]))  # rows 0, 1, 5 and 6 are nobody's
    out = torch.full_like(c.q, 7.0)
    binding.dspark_kv4_append_rotated(c.cache, c.batch, c.rotation, c.k, c.v, c.q, out)
    assert (out[[0, 1, 5, 6]] == 7).all() and not (out[2:5] == 7).all(2).any()


def test_captured_and_replayed_with_new_inputs():
    c = Rotated(rows=[6, 9], lens=[50, 9], page=16, heads=2, dim=64, q_heads=6)
    out, k = torch.empty_like(c.q), c.k.clone()
    c.k.zero_()
    binding.dspark_kv4_append_rotated(c.cache, c.batch, c.rotation, c.k, c.v, c.q, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.dspark_kv4_append_rotated(c.cache, c.batch, c.rotation, c.k, c.v, c.q, out)
    c.k.copy_(k)
    graph.replay()
    torch.cuda.synchronize()
    c.wants()
    same_bytes(c)


def test_on_another_stream():
    c = Rotated(rows=[6, 9], lens=[50, 9], page=16, heads=2, dim=64, q_heads=6)
    out, k, s = torch.empty_like(c.q), c.k.clone(), torch.cuda.Stream()
    c.k.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # the keys come late: on another stream the call would not see them
        c.k.copy_(k)
    binding.dspark_kv4_append_rotated(c.cache, c.batch, c.rotation, c.k, c.v, c.q, out, stream=s)
    torch.cuda.synchronize()
    want = c.wants()
    same_bytes(c)
    assert np.array_equal(out.float().cpu().numpy(), torch.from_numpy(want).to(c.q.dtype).float().numpy())
