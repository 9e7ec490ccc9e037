"""The entry points of include/dspark_kv4.h refuse bad arguments before any
CUDA call, and return at once where there is nothing to do (no GPU needed: the
pointers below are never followed)."""
import ctypes
import shutil
import os

import numpy as np
import pytest

from dspark_markov_draft_anchor_gb300 import binding, build
from tests import kv4_ref

INVALID, MISALIGNED, TOO_MANY = -1, -3, -4
AT = 1 << 20  # an aligned address


@pytest.fixture(scope="module")
def lib():
    if not build.up_to_date() and not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("nvcc not available to build the library")
    build.build()
    return binding.load()


def cache(**kw):
    c = dict(data=AT, page_stride=16 * 72 * 2, num_pages=4, page_size=16, kv_heads=2, head_dim=64, k_scale=None,
             v_scale=None)
    c.update(kw)
    return binding.Kv4CacheStruct(**c)


def batch(**kw):
    b = dict(batch=2, total_rows=3, max_rows=2, max_pages=4, max_slots=2, reserved=0, row_start=AT, slots=None,
             lens=AT, table=AT, table_stride=4)
    b.update(kw)
    return binding.Kv4BatchStruct(**b)


BAD_CACHES = [
    (dict(page_size=24), INVALID), (dict(page_size=8), INVALID), (dict(page_size=512), INVALID),
    (dict(head_dim=96), INVALID), (dict(head_dim=256), INVALID), (dict(kv_heads=0), INVALID),
    (dict(num_pages=-1), INVALID), (dict(page_stride=16 * 72 * 2 - 16), INVALID), (dict(data=None), INVALID),
    (dict(data=AT + 8), MISALIGNED), (dict(page_stride=16 * 72 * 2 + 8), MISALIGNED), (dict(k_scale=AT + 2), MISALIGNED),
]
BAD_BATCHES = [
    (dict(batch=-1), INVALID), (dict(total_rows=-1), INVALID), (dict(max_pages=5), INVALID), (dict(max_rows=-1), INVALID),
    (dict(max_slots=-1), INVALID), (dict(row_start=None), INVALID), (dict(lens=None), INVALID),
    (dict(table=None), INVALID), (dict(batch=binding.KV4_MAX_BATCH + 1), TOO_MANY), (dict(lens=AT + 1), MISALIGNED),
]


def every_call(lib, c, b):
    ref = lambda s: None if s is None else ctypes.addressof(s)  # noqa: E731
    a = binding.Kv4AttentionArgs(AT, 256, 64, AT, 256, 64, None, 4, 0, 0.1, 0, AT, 1 << 40)
    return [lib.dspark_kv4_append(ref(c), ref(b), AT, 128, 64, AT, 128, 64, 0, None),
            lib.dspark_kv4_read(ref(c), ref(b), AT, 128, 64, AT, 128, 64, 2, None),
            lib.dspark_kv4_attention(ref(c), ref(b), ctypes.addressof(a), None)]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches(lib, kw, want):
    c, b = cache(**kw), batch()
    assert every_call(lib, c, b) == [want] * 3
    assert lib.dspark_kv4_attention_workspace_bytes(ctypes.addressof(c), ctypes.addressof(b), 4) == 0


@pytest.mark.parametrize("kw,want", BAD_BATCHES)
def test_bad_batches(lib, kw, want):
    assert every_call(lib, cache(), batch(**kw)) == [want] * 3


def test_null_structures_and_empty_batches(lib):
    assert every_call(lib, None, batch()) == [INVALID] * 3
    assert every_call(lib, cache(), None) == [INVALID] * 3
    assert every_call(lib, cache(), batch(batch=0, row_start=None, lens=None, table=None)) == [0] * 3
    assert every_call(lib, cache(), batch(total_rows=0)) == [0] * 3


def test_rows_and_types(lib):
    c, b = cache(), batch()
    ap = lambda *a: lib.dspark_kv4_append(ctypes.addressof(c), ctypes.addressof(b), *a, None)  # noqa: E731
    assert ap(AT, 128, 64, AT, 128, 64, 2) == INVALID      # float32 is for reading
    assert ap(AT, 128, 64, AT, 128, 64, 7) == INVALID
    assert ap(None, 128, 64, AT, 128, 64, 0) == INVALID
    assert ap(AT, 128, 64, None, 128, 64, 0) == INVALID
    assert ap(AT, -1, 64, AT, 128, 64, 0) == INVALID
    assert ap(AT + 1, 128, 64, AT, 128, 64, 0) == MISALIGNED
    rd = lambda *a: lib.dspark_kv4_read(ctypes.addressof(c), ctypes.addressof(b), *a, None)  # noqa: E731
    assert rd(AT + 2, 128, 64, None, 0, 0, 2) == MISALIGNED
    assert rd(None, 0, 0, None, 0, 0, 0) == 0
    assert rd(AT, 128, 64, AT, 128, -2, 0) == INVALID


def test_attention_arguments(lib):
    c, b = cache(), batch()
    size = lib.dspark_kv4_attention_workspace_bytes(ctypes.addressof(c), ctypes.addressof(b), 4)
    assert size > 0

    def at(**kw):
        a = dict(q=AT, q_row=256, q_head=64, out=AT, out_row=256, out_head=64, lse=None, q_heads=4, dtype=0, scale=0.1,
                 window=0, workspace=AT, workspace_bytes=size)
        a.update(kw)
        a = binding.Kv4AttentionArgs(**a)
        return lib.dspark_kv4_attention(ctypes.addressof(c), ctypes.addressof(b), ctypes.addressof(a), None)
    for kw in (dict(q=None), dict(out=None), dict(workspace=None), dict(workspace_bytes=size - 1), dict(q_heads=3),
               dict(q_heads=0), dict(dtype=2), dict(window=-1), dict(scale=float("nan")), dict(scale=float("-inf")),
               dict(q_row=-1), dict(out_head=-1)):
        assert at(**kw) == INVALID, kw
    for kw in (dict(q=AT + 1), dict(out=AT + 1), dict(lse=AT + 2), dict(workspace=AT + 128)):
        assert at(**kw) == MISALIGNED, kw
    assert lib.dspark_kv4_attention(ctypes.addressof(c), ctypes.addressof(b), None, None) == INVALID


def pool(**kw):
    p = dict(num_pages=10, page_size=16, max_slots=4, max_pages=3, refs=AT, table=AT, table_stride=3, lens=AT)
    p.update(kw)
    return binding.PagePoolStruct(**p)


def page_calls(lib, p, n=2):
    r = None if p is None else ctypes.addressof(p)
    return [lib.dspark_pages_trim(r, n, AT, AT, None), lib.dspark_pages_fork(r, n, AT, AT, None),
            lib.dspark_pages_grow(r, n, AT, AT, AT, AT, AT, None)]


@pytest.mark.parametrize("kw,want", [
    (dict(num_pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(max_slots=-1), INVALID),
    (dict(table_stride=2), INVALID), (dict(refs=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(refs=AT + 2), MISALIGNED), (dict(lens=AT + 1), MISALIGNED)])
def test_bad_pools(lib, kw, want):
    assert page_calls(lib, pool(**kw)) == [want] * 3
    p = pool(**kw)
    assert lib.dspark_pages_compact(ctypes.addressof(p), AT, AT, AT, AT, AT, AT, None) == want


def test_page_lists(lib):
    p = pool()
    r = ctypes.addressof(p)
    assert page_calls(lib, None) == [INVALID] * 3
    assert page_calls(lib, p, -1) == [INVALID] * 3
    assert page_calls(lib, p, 0) == [0] * 3
    assert page_calls(lib, p, binding.PAGES_MAX_SLOTS + 1) == [TOO_MANY] * 3
    assert lib.dspark_pages_trim(r, 1, None, AT, None) == INVALID
    assert lib.dspark_pages_fork(r, 1, AT, None, None) == INVALID
    assert lib.dspark_pages_fork(r, 1, AT, AT + 2, None) == MISALIGNED
    assert lib.dspark_pages_grow(r, 1, AT, AT, None, AT, AT, None) == INVALID
    assert lib.dspark_pages_grow(r, 1, AT, AT, AT, AT + 1, AT, None) == MISALIGNED
    assert lib.dspark_pages_compact(r, AT, AT, AT, AT, AT, None, None) == INVALID
    assert lib.dspark_pages_compact(r, None, AT, AT, AT, AT, AT, None) == INVALID


def test_page_copies(lib):
    def cp(data=AT, pages=4, size=32, stride=32, layers=2, layer=128, n=1, src=AT, dst=AT, count=None):
        return lib.dspark_pages_copy(data, pages, size, stride, layers, layer, n, src, dst, count, None)
    for kw in (dict(pages=-1), dict(size=-16), dict(stride=16), dict(layers=-1), dict(layer=-16), dict(n=-1),
               dict(data=None), dict(src=None), dict(dst=None)):
        assert cp(**kw) == INVALID, kw
    for kw in (dict(data=AT + 8), dict(size=24), dict(stride=40), dict(layer=24), dict(src=AT + 1), dict(count=AT + 3)):
        assert cp(**kw) == MISALIGNED, kw
    for kw in (dict(n=0), dict(layers=0), dict(size=0), dict(pages=0)):
        assert cp(**kw) == 0, kw


# ---- the restatement that the GPU tests compare with ---------------------------

def test_restated_grids_are_the_formats():
    torch = pytest.importorskip("torch")
    bytes_ = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = bytes_.view(torch.float8_e4m3fn).float().numpy()
    nan = np.isnan(want)
    assert nan.sum() == 2 and np.array_equal(kv4_ref.E4M3[~nan], want[~nan]) and np.all(kv4_ref.E4M3[nan] == 448)
    x = np.concatenate([np.random.default_rng(0).random(20000) * 460, (kv4_ref.POSITIVE[1:] + kv4_ref.POSITIVE[:-1]) / 2])
    x = np.minimum(x, 448.0)
    code = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv4_ref.nearest(kv4_ref.POSITIVE, x.astype(np.float32).astype(np.float64)), code)


def test_restated_codes_are_nearest_with_ties_to_even():
    x = np.array([0, .25, .2500001, .75, .7499999, 1.25, 1.2500001, 1.75, 1.7499999, 2.5, 2.6, 3.5, 3.4, 5, 5.1, 6, 6.0])
    assert kv4_ref.nearest(kv4_ref.E2M1, x).tolist() == [0, 0, 1, 2, 1, 2, 3, 4, 3, 4, 5, 6, 5, 6, 7, 7, 7]
    y = np.zeros((1, 16))
    y[0, :4] = [6.0, -0.25, 1.25, -5.0]
    code, scale = kv4_ref.quantise(y, 1.0)
    assert kv4_ref.POSITIVE[scale] == 1.0 and code[0, :4].tolist() == [7, 8, 2, 14]
    assert np.array_equal(kv4_ref.values(code, scale, 1.0)[0, :4], [6.0, 0.0, 1.0, -4.0])
