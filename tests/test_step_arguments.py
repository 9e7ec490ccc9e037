"""The entry points for rotated appends, selections, token tables and adjusted logits refuse bad arguments before any
CUDA call and return at once where there is nothing to do, and the binding refuses tensors that are not laid out as the
kernels read them (no GPU needed: the pointers below are never followed)."""
import ctypes
import os
import shutil

import pytest

from dspark_markov_draft_anchor_gb300 import binding, build
from tests.test_kv4_arguments import AT, BAD_BATCHES, BAD_CACHES, INVALID, MISALIGNED, TOO_MANY, batch, cache

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    if not build.up_to_date() and not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("nvcc not available to build the library")
    build.build()
    return binding.load()


def ref(s):
    return None if s is None else ctypes.byref(s)  # keeps it alive


def make(kind, base, kw):
    return kind(**{**base, **kw})


ROTATION = dict(cos=AT, sin=AT, stride=32, positions=100, dims=64, interleaved=0, reserved=0, at=None)
ROTATED = dict(k=AT, k_row=128, k_head=64, v=AT, v_row=128, v_head=64, q=AT, q_row=256, q_head=64, q_out=AT + 4096,
               out_row=256, out_head=64, q_heads=4, dtype=0)
SELECTION = dict(pages=AT, lens=AT, rows=3, top=3)
SELECT = dict(q=AT, q_row=256, q_head=64, q_heads=4, dtype=0, first=1, last=2, workspace=AT, workspace_bytes=1 << 40)
ATTEND = dict(q=AT, q_row=256, q_head=64, out=AT, out_row=256, out_head=64, lse=None, q_heads=4, dtype=0, scale=0.1,
              window=0, workspace=AT, workspace_bytes=1 << 40)
BOUNDS = 2 * (2 * 64 + 16)


def rotated(lib, c=None, b=None, rotation=None, args=None):
    return lib.dspark_kv4_append_rotated(ref(c or cache()), ref(b or batch()),
                                         ref(make(binding.Kv4RotationStruct, ROTATION, rotation or {})),
                                         ref(make(binding.Kv4RotatedArgs, ROTATED, args or {})), None)


def bound(lib, c=None, b=None, bounds=AT, stride=BOUNDS):
    return lib.dspark_kv4_bound_pages(ref(c or cache()), ref(b or batch()), bounds, stride, None)


def select(lib, c=None, b=None, bounds=AT, stride=BOUNDS, selection=None, args=None):
    return lib.dspark_kv4_select(ref(c or cache()), ref(b or batch()), bounds, stride,
                                 ref(make(binding.Kv4SelectionStruct, SELECTION, selection or {})),
                                 ref(make(binding.Kv4SelectArgs, SELECT, args or {})), None)


def attend(lib, c=None, selection=None, args=None):
    return lib.dspark_kv4_attention_selected(ref(c or cache()),
                                             ref(make(binding.Kv4SelectionStruct, SELECTION, selection or {})),
                                             ref(make(binding.Kv4AttentionArgs, ATTEND, args or {})), None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches(lib, kw, want):
    c = cache(**kw)
    # a short page stride may be a bad stride, whatever the order of the checks
    assert [rotated(lib, c), bound(lib, c), select(lib, c), attend(lib, c)] == [want] * 4


@pytest.mark.parametrize("kw,want", BAD_BATCHES)
def test_bad_batches(lib, kw, want):
    b = batch(**kw)
    assert [rotated(lib, b=b), bound(lib, b=b), select(lib, b=b)] == [want] * 3


def test_rotation(lib):
    for kw in (dict(dims=0), dict(dims=16), dict(dims=48), dict(dims=96), dict(dims=128), dict(positions=-1),
               dict(stride=31), dict(cos=None), dict(sin=None)):
        assert rotated(lib, rotation=kw) == INVALID, kw
    for kw in (dict(cos=AT + 2), dict(sin=AT + 1), dict(at=AT + 2)):
        assert rotated(lib, rotation=kw) == MISALIGNED, kw
    for kw in (dict(k=None), dict(v=None), dict(q=None), dict(q_out=None), dict(dtype=2), dict(dtype=-1), dict(k_row=-1),
               dict(v_head=-1), dict(q_row=-1), dict(out_head=-1), dict(q_heads=0), dict(q_out=AT, out_row=512),
               dict(q_out=AT, out_head=128), dict(q_heads=2 ** 31 - 4)):
        assert rotated(lib, args=kw) == INVALID, kw
    for kw in (dict(k=AT + 1), dict(q=AT + 1), dict(q_out=AT + 1)):
        assert rotated(lib, args=kw) == MISALIGNED, kw
    assert lib.dspark_kv4_append_rotated(ref(cache()), ref(batch()), None, None, None) == INVALID
    assert rotated(lib, b=batch(total_rows=0)) == 0 and rotated(lib, b=batch(batch=0)) == 0


def test_bounds_and_selection(lib):
    for kw in (dict(bounds=None), dict(stride=BOUNDS - 16)):
        assert bound(lib, **kw) == INVALID and select(lib, **kw) == INVALID, kw
    for kw in (dict(bounds=AT + 8), dict(stride=BOUNDS + 8)):
        assert bound(lib, **kw) == MISALIGNED and select(lib, **kw) == MISALIGNED, kw
    for kw in (dict(top=0), dict(rows=-1), dict(pages=None), dict(lens=None)):
        assert select(lib, selection=kw) == INVALID and attend(lib, selection=kw) == INVALID, kw
    for kw in (dict(pages=AT + 2), dict(lens=AT + 1)):
        assert select(lib, selection=kw) == MISALIGNED and attend(lib, selection=kw) == MISALIGNED, kw
    assert select(lib, selection=dict(rows=2)) == INVALID  # rows of the batch are wanted
    for kw in (dict(q=None), dict(workspace=None), dict(workspace_bytes=100), dict(q_heads=3), dict(q_heads=0),
               dict(dtype=2), dict(q_row=-1), dict(first=-1), dict(last=0), dict(first=2), dict(last=3),
               dict(first=2 ** 31 - 1), dict(last=2 ** 31 - 1)):
        assert select(lib, args=kw) == INVALID, kw
    for kw in (dict(q=AT + 1), dict(workspace=AT + 128)):
        assert select(lib, args=kw) == MISALIGNED, kw
    assert bound(lib, b=batch(total_rows=0)) == 0
    assert select(lib, b=batch(total_rows=0), selection=dict(rows=0)) == 0
    c, b, s = cache(), batch(), binding.Kv4SelectionStruct(**SELECTION)
    # 3 rows of 2 heads: keys of 4 pages and 128 bytes of parts each
    assert lib.dspark_kv4_select_workspace_bytes(ref(c), ref(b), ref(s)) == 6 * (16 + 128) + 256
    assert lib.dspark_kv4_select_workspace_bytes(ref(c), ref(b), None) == 0
    assert lib.dspark_kv4_select_workspace_bytes(ref(c), ref(batch(max_pages=3)), ref(s)) == 256


def test_attention_selected(lib):
    for kw in (dict(q=None), dict(out=None), dict(workspace=None), dict(workspace_bytes=100), dict(q_heads=3),
               dict(dtype=2), dict(window=1), dict(window=-1), dict(scale=float("inf")), dict(q_row=-1), dict(out_row=-1)):
        assert attend(lib, args=kw) == INVALID, kw
    for kw in (dict(q=AT + 1), dict(out=AT + 1), dict(lse=AT + 2), dict(workspace=AT + 128)):
        assert attend(lib, args=kw) == MISALIGNED, kw
    assert attend(lib, selection=dict(rows=0, pages=None, lens=None)) == 0
    assert lib.dspark_kv4_attention_selected(ref(cache()), None, None, None) == INVALID
    size = lib.dspark_kv4_attention_selected_workspace_bytes
    s = binding.Kv4SelectionStruct(**SELECTION)
    assert size(ref(cache()), ref(s), 4) > 0 and size(ref(cache()), ref(s), 3) == 0 and size(None, ref(s), 4) == 0
    assert size(ref(cache()), None, 4) == 0


TABLE = dict(counts=AT, counts_stride=100, marks=AT, marks_stride=8, vocab=100, max_slots=3)
ADJUST = dict(logits=AT, logits_stride=100, out=AT + 65536, out_stride=100, dtype=0, out_dtype=2, batch=2, drafts=1,
              vocab=100, max_slots=3, slots=None, draft=AT, draft_stride=1, repetition=AT, frequency=AT, presence=AT,
              bias_start=AT, bias_id=AT, bias=AT, bias_entries=5, mask=AT, mask_stride=4, mask_rows=4, mask_row=AT)


def count(lib, table=None, n=2, slots=AT, tokens=AT, wide=1, stride=5, width=5, lens=AT):
    return lib.dspark_tokens_count(ref(make(binding.TokenTableStruct, TABLE, table or {})), n, slots, tokens, wide,
                                   stride, width, lens, 0, 1, None)


def adjust(lib, table=None, **kw):
    t = make(binding.TokenTableStruct, TABLE, table or {})
    return lib.dspark_logits_adjust(ref(t), ref(make(binding.AdjustArgs, ADJUST, kw)), None)


def test_token_tables(lib):
    for kw in (dict(counts=None), dict(marks=None), dict(counts_stride=99), dict(marks_stride=7), dict(vocab=0),
               dict(vocab=2 ** 30 + 1), dict(max_slots=-1)):
        assert count(lib, kw) == INVALID and adjust(lib, kw) == INVALID, kw
    for kw in (dict(counts=AT + 2), dict(marks=AT + 1)):
        assert count(lib, kw) == MISALIGNED and adjust(lib, kw) == MISALIGNED, kw
    for kw in (dict(n=-1), dict(width=-1), dict(stride=4), dict(lens=None), dict(tokens=None)):
        assert count(lib, **kw) == INVALID, kw
    for kw in (dict(tokens=AT + 4), dict(tokens=AT + 2, wide=0), dict(lens=AT + 2), dict(slots=AT + 1)):
        assert count(lib, **kw) == MISALIGNED, kw
    assert count(lib, n=0) == 0 and count(lib, dict(max_slots=0, counts=None, marks=None)) == 0
    assert lib.dspark_tokens_count(None, 1, AT, AT, 1, 5, 5, AT, 0, 0, None) == INVALID


def test_adjust(lib):
    for kw in (dict(logits=None), dict(out=None), dict(logits_stride=99), dict(out_stride=99), dict(dtype=1),
               dict(out_dtype=1), dict(dtype=2, out_dtype=0), dict(batch=-1), dict(drafts=-1), dict(vocab=0),
               dict(vocab=101, logits_stride=101, out_stride=101), dict(max_slots=2), dict(draft=None),
               dict(draft_stride=0), dict(bias_start=None), dict(bias_id=None), dict(bias=None), dict(bias_entries=-1),
               dict(mask_stride=3), dict(mask_rows=-1), dict(out=AT), dict(out=AT, out_dtype=0, out_stride=104)):
        assert adjust(lib, **kw) == INVALID, kw
    assert adjust(lib, drafts=1024, draft_stride=1024) == TOO_MANY
    for kw in (dict(logits=AT + 1), dict(out=AT + 65538), dict(draft=AT + 4), dict(mask=AT + 2), dict(bias=AT + 1),
               dict(repetition=AT + 2), dict(slots=AT + 1), dict(mask_row=AT + 3)):
        assert adjust(lib, **kw) == MISALIGNED, kw
    assert adjust(lib, batch=0) == 0
    assert lib.dspark_logits_adjust(None, None, None) == INVALID


# ---- the binding ---------------------------------------------------------------

def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


I = torch.int32  # noqa: E741


def step(rows=3, heads=2, dim=64):
    c = binding.Kv4Cache(z(4, binding.kv4_page_bytes(16, heads, dim), dtype=torch.uint8), 16, heads, dim)
    b = binding.Kv4Batch(torch.tensor([0, rows], dtype=I), torch.tensor([rows], dtype=I), z(1, 4, dtype=I),
                         total_rows=rows, max_rows=rows)
    return c, b


def rows(heads=2, n=3, dim=64, dtype=torch.bfloat16):
    return z(n, heads, dim, dtype=dtype)


def test_rotation_tables_are_refused():
    for cos, sin in ((z(9, 32, dtype=torch.float64), z(9, 32)), (z(9, 32), z(9, 31)), (z(9, 32), z(9, 64)[:, ::2]),
                     (z(9, 32), z(9, 40)[:, :32]), (z(1, 32).expand(9, 32), z(1, 32).expand(9, 32)), (z(32), z(32))):
        with pytest.raises((ValueError, TypeError)):
            binding.Kv4Rotation(cos, sin)
    with pytest.raises(TypeError):
        binding.Kv4Rotation(z(9, 32), z(9, 32), positions=z(3))
    wide = z(9, 80)
    assert binding.Kv4Rotation(wide[:, :32], wide[:, 40:72]).struct.stride == 80


def test_rotated_rows_are_refused():
    c, b = step()
    r = binding.Kv4Rotation(z(9, 32), z(9, 32))
    short = binding.Kv4Rotation(z(9, 32), z(9, 32), positions=z(2, dtype=I))
    q = rows(4)
    for rot, args in ((r, (rows(), rows(), q)), (r, (rows(), rows(), None, q)), (r, (rows(), rows(n=2), q, q)),
                      (r, (rows(), rows(3), q, q)), (r, (rows(), rows(dtype=torch.float16), q, q)),
                      (r, (rows(), rows(), q, rows(5))), (r, (rows(), rows(), q, q.half())),
                      (r, (rows(), rows(dim=128), q, q)), (short, (rows(), rows(), q, q)),
                      (r, (rows(), rows(), q, q))):  # the last: not on a GPU
        with pytest.raises((ValueError, TypeError)):
            binding.dspark_kv4_append_rotated(c, b, rot, *args)


def test_selections_are_refused():
    c, b = step()
    for pages, lens in ((z(3, 2, 4), z(3, dtype=I)), (z(3, 2, 4, dtype=I), z(2, dtype=I)), (z(3, 8, dtype=I), z(3, dtype=I)),
                        (z(3, 2, 8, dtype=I)[:, :, ::2], z(3, dtype=I)), (z(3, 2, 4, dtype=I), z(3, 1, dtype=I))):
        with pytest.raises((ValueError, TypeError)):
            binding.Kv4Selection(pages, lens)
    good = binding.Kv4Selection(z(3, 2, 4, dtype=I), z(3, dtype=I))
    other = binding.Kv4Selection(z(3, 5, 4, dtype=I), z(3, dtype=I))
    bounds, ws, q = z(4, binding.kv4_bounds_bytes(2, 64), dtype=torch.uint8), z(1 << 20, dtype=torch.uint8), rows(4)
    for args in ((bounds, q, other, ws), (bounds[:3], q, good, ws), (bounds[:, :100], q, good, ws), (bounds.int(), q, good, ws),
                 (bounds, rows(4, 2), good, ws), (bounds, rows(4, dim=128), good, ws), (bounds, q, good, ws)):
        with pytest.raises((ValueError, TypeError)):
            binding.dspark_kv4_select(c, b, *args)
    for sel, x, y, kw in ((other, q, q, {}), (good, rows(4, 2), q, {}), (good, q, rows(5), {}), (good, q, q.half(), {}),
                          (good, q, q, dict(lse=z(3, 5))), (good, q, q, dict(lse=z(3, 4, dtype=torch.bfloat16))), (good, q, q, {})):
        with pytest.raises((ValueError, TypeError)):
            binding.dspark_kv4_attention_selected(c, sel, x, y, 1.0, ws, **kw)
    with pytest.raises((ValueError, TypeError)):
        binding.dspark_kv4_bound_pages(c, b, bounds)  # not on a GPU


def test_token_tables_and_tokens_are_refused():
    for counts, marks in ((z(2, 40), z(2, 2, 2, dtype=I)), (z(2, 40, dtype=I), z(2, 2, 1, dtype=I)),
                          (z(2, 40, dtype=I), z(3, 2, 2, dtype=I)), (z(2, 40, dtype=I), z(2, 2, 4, dtype=I)[:, :, ::2]),
                          (z(1, 40, dtype=I).expand(2, 40), z(2, 2, 2, dtype=I)), (z(2, 80, dtype=I)[:, ::2], z(2, 2, 2, dtype=I)),
                          (z(2, 40, dtype=I), z(1, 2, 2, dtype=I).expand(2, 2, 2)), (z(2, 40, dtype=I), z(2, 2, 2))):
        with pytest.raises((ValueError, TypeError)):
            binding.TokenTable(counts, marks)
    t = binding.TokenTable(z(2, 40, dtype=I), z(2, 3, 2, dtype=I)[:, :2])
    assert t.struct.marks_stride == 6
    tokens, lens = z(2, 5, dtype=torch.int64), z(2, dtype=I)
    for args, kw in (((tokens.float(), lens), {}), ((tokens, z(3, dtype=I)), {}), ((tokens, lens.long()), {}),
                     ((tokens[:, ::2], lens), {}), ((tokens[0], lens), {}), ((tokens, lens), dict(slots=z(3, dtype=I))),
                     ((tokens, lens), dict(slots=lens.long())), ((tokens, lens), {})):
        with pytest.raises((ValueError, TypeError)):
            binding.dspark_tokens_count(t, *args, **kw)


def test_logits_are_refused(monkeypatch):
    monkeypatch.setattr(binding, "_on_one_device", lambda *a: None)  # what is refused beside that
    monkeypatch.setattr(binding, "load", lambda: pytest.fail("the library was called"))
    t = binding.TokenTable(z(2, 40, dtype=I), z(2, 2, 2, dtype=I))
    x, y = z(4, 40, dtype=torch.bfloat16), z(4, 40)
    good = dict(drafts=1, draft=z(2, 1, dtype=torch.int64))
    for args, kw in (((x, z(3, 40)), {}), ((x, z(4, 41)), {}), ((x.T, y.T), {}), ((x[:1].expand(4, 40), y), {}),
                     ((x, y[:1].expand(4, 40)), {}), ((x, y), dict(drafts=2)), ((x, y), dict(drafts=-1)),
                     ((x, y), dict(drafts=-2)), ((x, y), dict(draft=z(2, 1))), ((x, y), dict(draft=z(3, 1, dtype=torch.int64))),
                     ((x, y), dict(draft=z(2, 2, dtype=torch.int64))), ((x, y), dict(slots=z(3, dtype=I))),
                     ((x, y), dict(slots=z(2))), ((x, y), dict(repetition=z(3))), ((x, y), dict(frequency=z(2, dtype=torch.float64))),
                     ((x, y), dict(presence=z(4)[::2])), ((x, y), dict(bias=(z(2, dtype=I), z(5, dtype=I), z(5)))),
                     ((x, y), dict(bias=(z(3, dtype=I), z(5, dtype=I), z(4)))), ((x, y), dict(bias=(z(3, dtype=I), z(5), z(5)))),
                     ((x, y), dict(mask=z(4, 1, dtype=I))), ((x, y), dict(mask=z(4, 2))), ((x, y), dict(mask=z(4, 4, dtype=I)[:, ::2])),
                     ((x, y), dict(mask=z(1, 2, dtype=I).expand(4, 2))), ((x, y), dict(mask=z(4, 2, dtype=I), mask_rows=z(3, dtype=I))),
                     ((x, y), dict(mask_rows=z(3, dtype=I)))):
        with pytest.raises((ValueError, TypeError)):
            binding.dspark_logits_adjust(t, *args, **{**good, **kw})


def test_logits_elsewhere_are_refused():
    with pytest.raises(ValueError):
        binding.dspark_logits_adjust(None, z(4, 40), z(4, 40))
