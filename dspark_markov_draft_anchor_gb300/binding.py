"""ctypes binding of libdspark_markov.so (argument marshalling only).

The functions here carry the C ABI's names and forward to it; every step of
the loop runs in the library's CUDA kernels.  torch tensors are accepted for
convenience (their data pointers and strides are passed through).  There is
no fallback: if the library is missing or the device is not a GB300, calls
raise.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

DSPARK_OK = 0
ERRORS = {
    -1: "DSPARK_ERR_INVALID_ARG", -2: "DSPARK_ERR_UNSUPPORTED_RANK", -3: "DSPARK_ERR_MISALIGNED",
    -4: "DSPARK_ERR_TOO_MANY_ROWS", -5: "DSPARK_ERR_CAPTURING", -6: "DSPARK_ERR_CUDA",
    -7: "DSPARK_ERR_DEVICE_TIMEOUT", -8: "DSPARK_ERR_UNSUPPORTED_DEVICE", -9: "DSPARK_ERR_HOST_ALLOC",
}
FLAG_PDL = 0x1
FLAG_FORCE_FMA = 0x2
FLAG_FORCE_MMA = 0x4
FLAG_PER_STEP = 0x8
FLAG_SELECT_2LAUNCH = 0x10
FLAG_TEST_STALL = 0x100
NOALLOC_MAX_VERIFY_ROWS = 8192  # DSPARK_NOALLOC_MAX_VERIFY_ROWS

EXPORTED = (
    "dspark_markov_init", "dspark_markov_loop", "dspark_markov_anchor", "dspark_markov_step",
    "dspark_markov_partial_count", "dspark_markov_bias_path", "dspark_markov_set_w2_fp8", "dspark_markov_loop_kernels",
    "dspark_markov_get_status",
    "dspark_markov_get_status_detail",
    "dspark_markov_destroy", "dspark_build_verify_tokens", "dspark_greedy_accept_scratch_bytes",
    "dspark_greedy_accept", "dspark_greedy_accept_noalloc", "dspark_fill_uniforms",
    "dspark_probabilistic_accept", "dspark_logits_to_probs", "dspark_quantize_w2_fp8", "dspark_strerror",
    "dspark_check_noise_range", "dspark_check_hash", "dspark_check_logit", "dspark_check_key",
    "dspark_check_logf", "dspark_check_tanhf", "dspark_check_expf", "dspark_check_div",
    "dspark_check_div_sweep", "dspark_noise_bound_tables",
    "dspark_markov_shard_step", "dspark_markov_pick", "dspark_cache_fill",
    "dspark_confidence_scores", "dspark_confidence_and_proposal_lengths",
    "dspark_confidence_and_sps_proposal_lengths",
    "dspark_kv4_append", "dspark_kv4_read", "dspark_kv4_attention_workspace_bytes", "dspark_kv4_attention",
    "dspark_pages_trim", "dspark_pages_fork", "dspark_pages_grow", "dspark_pages_compact", "dspark_pages_copy",
)
DTYPE_BF16, DTYPE_F16, DTYPE_F32 = 0, 1, 2  # DSPARK_DTYPE_*
KV4_MAX_BATCH = 4096  # DSPARK_KV4_MAX_BATCH
PAGES_MAX_SLOTS = 4096  # DSPARK_PAGES_MAX_SLOTS
CONFIDENCE_MAX_P = 256  # DSPARK_CONFIDENCE_MAX_P


class DsparkError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {ERRORS.get(code, code)} ({strerror(code)})")


class MarkovConfig(ctypes.Structure):
    _fields_ = [("vocab", ctypes.c_int32), ("rank", ctypes.c_int32), ("w1_rows", ctypes.c_int32),
                ("max_rows", ctypes.c_int32), ("max_steps", ctypes.c_int32), ("flags", ctypes.c_int32)]


class ConfidenceArgs(ctypes.Structure):
    _fields_ = [
        ("hidden", ctypes.c_void_p), ("hidden_stride", ctypes.c_int64), ("hidden_offset", ctypes.c_int64),
        ("hidden_size", ctypes.c_int32), ("with_markov", ctypes.c_int32),
        ("w1", ctypes.c_void_p), ("w1_rows", ctypes.c_int64), ("rank", ctypes.c_int32),
        ("batch", ctypes.c_int32), ("proposal_len", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("first_prev", ctypes.c_void_p),
        ("draft", ctypes.c_void_p), ("draft_s0", ctypes.c_int64),
        ("scores", ctypes.c_void_p), ("logits", ctypes.c_void_p),
    ]


class LoopArgs(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32), ("steps", ctypes.c_int32),
        ("base", ctypes.c_void_p), ("base_s0", ctypes.c_int64), ("base_s1", ctypes.c_int64),
        ("cache", ctypes.c_void_p), ("cache_s0", ctypes.c_int64), ("cache_s1", ctypes.c_int64),
        ("input_ids", ctypes.c_void_p), ("anchor_idx", ctypes.c_void_p),
        ("req_idx", ctypes.c_void_p), ("req_s0", ctypes.c_int64),
        ("sample_pos", ctypes.c_void_p), ("pos_s0", ctypes.c_int64),
        ("num_req", ctypes.c_int64), ("seeds", ctypes.c_void_p), ("temperature", ctypes.c_void_p),
        ("mult", ctypes.c_float), ("cap", ctypes.c_float), ("salt", ctypes.c_uint32),
        ("tokens", ctypes.c_void_p), ("tokens_s0", ctypes.c_int64),
        ("bias_out", ctypes.c_void_p),
    ]


class Kv4CacheStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class Kv4BatchStruct(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("total_rows", ctypes.c_int32), ("max_rows", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("max_slots", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("row_start", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64)]


class Kv4AttentionArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_row", ctypes.c_int64), ("out_head", ctypes.c_int64),
                ("lse", ctypes.c_void_p), ("q_heads", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("window", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class PagePoolStruct(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_slots", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("refs", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p)]


_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load(build_if_missing: bool = False):
    """Load libdspark_markov.so; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(f"{path} is missing: build it with dspark_markov_draft_anchor_gb300.build.build()")
        _build.build()
    L = ctypes.CDLL(path)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "dspark_markov_init": (ctypes.c_int, [ctypes.POINTER(P), ctypes.POINTER(MarkovConfig), P, P, P]),
        "dspark_markov_loop": (ctypes.c_int, [P, ctypes.POINTER(LoopArgs), P]),
        "dspark_markov_anchor": (ctypes.c_int, [P, ctypes.POINTER(LoopArgs), P]),
        "dspark_markov_step": (ctypes.c_int, [P, ctypes.POINTER(LoopArgs), i32, P]),
        "dspark_markov_partial_count": (i32, [P]),
        "dspark_markov_bias_path": (i32, [P, i32]),
        "dspark_markov_set_w2_fp8": (ctypes.c_int, [P, P, P]),
        "dspark_markov_loop_kernels": (i32, [P, ctypes.POINTER(LoopArgs)]),
        "dspark_markov_get_status": (ctypes.c_int, [P, P, ctypes.POINTER(i32)]),
        "dspark_markov_get_status_detail": (ctypes.c_int, [P, P, ctypes.POINTER(i32)]),
        "dspark_markov_destroy": (None, [P]),
        "dspark_build_verify_tokens": (ctypes.c_int, [P, P, P, i32, i32, i32, P]),
        "dspark_greedy_accept_scratch_bytes": (sz, [i32, i32, i32]),
        "dspark_greedy_accept": (ctypes.c_int, [P, P, P, P, P, P, sz, i32, i32, i32, i32, P]),
        "dspark_greedy_accept_noalloc": (ctypes.c_int, [P, P, P, P, P, i32, i32, i32, i32, P]),
        "dspark_fill_uniforms": (ctypes.c_int, [P, i64, ctypes.c_uint64, ctypes.c_uint64, P]),
        "dspark_probabilistic_accept": (ctypes.c_int, [P, P, P, P, P, P, P, i32, i32, i32, i32, P]),
        "dspark_logits_to_probs": (ctypes.c_int, [P, P, i32, i32, ctypes.c_float, i32, ctypes.c_float, P]),
        "dspark_quantize_w2_fp8": (ctypes.c_int, [P, P, P, i64, i32, P]),
        "dspark_strerror": (ctypes.c_char_p, [ctypes.c_int]),
        "dspark_check_noise_range": (ctypes.c_int, [ctypes.c_uint32, P, i64, P]),
        "dspark_check_hash": (ctypes.c_int, [i64, i32, i64, ctypes.c_uint32, P, P, i64, P]),
        "dspark_check_logit": (ctypes.c_int, [P, P, P, P, i64, ctypes.c_float, ctypes.c_float, P]),
        "dspark_check_key": (ctypes.c_int, [P, ctypes.c_float, P, P, i64, P]),
        "dspark_check_logf": (ctypes.c_int, [P, P, i64, P]),
        "dspark_check_tanhf": (ctypes.c_int, [P, P, i64, P]),
        "dspark_check_expf": (ctypes.c_int, [P, P, i64, P]),
        "dspark_check_div": (ctypes.c_int, [P, ctypes.c_float, P, i64, P]),
        "dspark_check_div_sweep": (ctypes.c_int, [ctypes.c_float, ctypes.c_uint32, i64, P, P]),
        "dspark_noise_bound_tables": (ctypes.c_int, [P, P, i32]),
        "dspark_markov_shard_step": (ctypes.c_int, [P, ctypes.POINTER(LoopArgs), i32, i64, P, P]),
        "dspark_markov_pick": (ctypes.c_int, [P, P, i32, i32, P, i64, i32, P]),
        "dspark_cache_fill": (ctypes.c_int, [P, i64, P, i64, i64, P, i64, i64, i32, i32, i32, i32, i32, P]),
        "dspark_confidence_scores": (ctypes.c_int, [ctypes.POINTER(ConfidenceArgs), P]),
        "dspark_confidence_and_proposal_lengths": (
            ctypes.c_int, [ctypes.POINTER(ConfidenceArgs), ctypes.c_float, i32, i32, P, P]),
        "dspark_confidence_and_sps_proposal_lengths": (
            ctypes.c_int, [ctypes.POINTER(ConfidenceArgs), ctypes.c_float, i32, i32, P, P, P]),
        "dspark_kv4_append": (ctypes.c_int, [P, P, P, i64, i64, P, i64, i64, i32, P]),
        "dspark_kv4_read": (ctypes.c_int, [P, P, P, i64, i64, P, i64, i64, i32, P]),
        "dspark_kv4_attention_workspace_bytes": (sz, [P, P, i32]),
        "dspark_kv4_attention": (ctypes.c_int, [P, P, P, P]),
        "dspark_pages_trim": (ctypes.c_int, [P, i32, P, P, P]),
        "dspark_pages_fork": (ctypes.c_int, [P, i32, P, P, P]),
        "dspark_pages_grow": (ctypes.c_int, [P, i32, P, P, P, P, P, P]),
        "dspark_pages_compact": (ctypes.c_int, [P, P, P, P, P, P, P, P]),
        "dspark_pages_copy": (ctypes.c_int, [P, i32, i64, i64, i32, i64, i32, P, P, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    _lib = L
    return L


def strerror(code: int) -> str:
    try:
        return load().dspark_strerror(code).decode()
    except Exception:  # library not loadable: still report the code
        return ERRORS.get(code, str(code))


def _check(rc: int, what: str):
    if rc != DSPARK_OK:
        raise DsparkError(rc, what)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_current_raw_stream = None


def _current_stream():
    """The current stream's handle (through torch's raw getter where there is
    one: building a Stream object costs as much as a launch)."""
    global _current_raw_stream
    if _current_raw_stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None or not torch.cuda.is_available():
            _current_raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        else:
            torch.cuda.init()
            device = torch.cuda.current_device
            _current_raw_stream = lambda: raw(device())  # noqa: E731
    return _current_raw_stream()


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# --------------------------------------------------------------------------
# C-ABI entry points
# --------------------------------------------------------------------------

def dspark_markov_init(vocab, rank, w1_rows, max_rows, max_steps, flags, w1, w2, stream=None):
    cfg = MarkovConfig(vocab, rank, w1_rows, max_rows, max_steps, flags)
    ctx = ctypes.c_void_p()
    _check(load().dspark_markov_init(ctypes.byref(ctx), ctypes.byref(cfg), _ptr(w1), _ptr(w2), _stream(stream)),
           "dspark_markov_init")
    return ctx


def dspark_markov_destroy(ctx):
    load().dspark_markov_destroy(ctx)


def dspark_markov_loop(ctx, args: LoopArgs, stream=None):
    _check(load().dspark_markov_loop(ctx, ctypes.byref(args), _stream(stream)), "dspark_markov_loop")


def dspark_markov_anchor(ctx, args: LoopArgs, stream=None):
    _check(load().dspark_markov_anchor(ctx, ctypes.byref(args), _stream(stream)), "dspark_markov_anchor")


def dspark_markov_step(ctx, args: LoopArgs, step: int, stream=None):
    _check(load().dspark_markov_step(ctx, ctypes.byref(args), step, _stream(stream)), "dspark_markov_step")


def dspark_markov_shard_step(ctx, args: LoopArgs, step: int, vocab_offset: int, packets, stream=None):
    """One step on a vocabulary shard; packets: int32 [rows, 4] (device)."""
    _check(load().dspark_markov_shard_step(ctx, ctypes.byref(args), step, vocab_offset, _ptr(packets),
                                           _stream(stream)), "dspark_markov_shard_step")


def dspark_markov_pick(ctx, packets, tp: int, rows: int, tokens, tokens_s0: int, step: int, stream=None):
    """The winners of the gathered packets int32 [tp, rows, 4] into tokens[:, step]."""
    _check(load().dspark_markov_pick(ctx, _ptr(packets), tp, rows, _ptr(tokens), tokens_s0, step, _stream(stream)),
           "dspark_markov_pick")


def dspark_cache_fill(src, src_s0: int, cache, cache_s0: int, cache_s1: int, req_idx, req_s0: int, num_req: int,
                      rows: int, steps: int, shard: int, tp: int, vocab: int, stream=None):
    _check(load().dspark_cache_fill(_ptr(src), src_s0, _ptr(cache), cache_s0, cache_s1, _ptr(req_idx), req_s0,
                                    num_req, rows, steps, shard, tp, vocab, _stream(stream)), "dspark_cache_fill")


def dspark_markov_partial_count(ctx) -> int:
    return int(load().dspark_markov_partial_count(ctx))


def dspark_markov_bias_path(ctx, rows: int) -> int:
    return int(load().dspark_markov_bias_path(ctx, rows))


def dspark_markov_set_w2_fp8(ctx, w2_fp8, w2_scale_f16):
    _check(load().dspark_markov_set_w2_fp8(ctx, _ptr(w2_fp8), _ptr(w2_scale_f16)), "dspark_markov_set_w2_fp8")


def dspark_markov_loop_kernels(ctx, args: LoopArgs) -> int:
    return int(load().dspark_markov_loop_kernels(ctx, ctypes.byref(args)))


def dspark_markov_get_status(ctx, stream=None) -> int:
    st = ctypes.c_int32(0)
    _check(load().dspark_markov_get_status(ctx, _stream(stream), ctypes.byref(st)), "dspark_markov_get_status")
    return int(st.value)


def dspark_markov_get_status_detail(ctx, stream=None) -> list:
    d = (ctypes.c_int32 * 4)()
    _check(load().dspark_markov_get_status_detail(ctx, _stream(stream), d), "dspark_markov_get_status_detail")
    return list(d)


def confidence_args(*, hidden, w1, weight, bias, first_prev, draft, scores, batch, proposal_len, hidden_size,
                    rank, w1_rows, with_markov=True, hidden_stride=0, hidden_offset=0, draft_s0=None,
                    logits=None) -> ConfidenceArgs:
    """Marshal device tensors (or raw addresses) into dspark_confidence_args."""
    if draft_s0 is None:
        draft_s0 = draft.stride(0) if hasattr(draft, "stride") else proposal_len
    return ConfidenceArgs(_ptr(hidden), hidden_stride, hidden_offset, hidden_size, int(bool(with_markov)),
                          _ptr(w1), w1_rows, rank, batch, proposal_len, 0, _ptr(weight), _ptr(bias),
                          _ptr(first_prev), _ptr(draft), draft_s0, _ptr(scores), _ptr(logits))


def dspark_confidence_scores(args: ConfidenceArgs, stream=None):
    _check(load().dspark_confidence_scores(ctypes.byref(args), _stream(stream)), "dspark_confidence_scores")


def dspark_confidence_and_proposal_lengths(args: ConfidenceArgs, threshold: float, min_proposal_len: int,
                                           max_proposal_len: int, proposal_lengths, stream=None):
    _check(load().dspark_confidence_and_proposal_lengths(ctypes.byref(args), threshold, min_proposal_len,
                                                         max_proposal_len, _ptr(proposal_lengths),
                                                         _stream(stream)),
           "dspark_confidence_and_proposal_lengths")


def dspark_confidence_and_sps_proposal_lengths(args: ConfidenceArgs, survival_floor: float, min_proposal_len: int,
                                               max_proposal_len: int, verify_cost, proposal_lengths, stream=None):
    _check(load().dspark_confidence_and_sps_proposal_lengths(ctypes.byref(args), survival_floor, min_proposal_len,
                                                             max_proposal_len, _ptr(verify_cost),
                                                             _ptr(proposal_lengths), _stream(stream)),
           "dspark_confidence_and_sps_proposal_lengths")


def dspark_build_verify_tokens(last, draft, verify, batch, draft_stride, P, stream=None):
    _check(load().dspark_build_verify_tokens(_ptr(last), _ptr(draft), _ptr(verify), batch, draft_stride, P,
                                             _stream(stream)), "dspark_build_verify_tokens")


def dspark_greedy_accept_scratch_bytes(batch, P, vocab) -> int:
    return int(load().dspark_greedy_accept_scratch_bytes(batch, P, vocab))


def dspark_greedy_accept(logits, draft, proposal_len, accepted, accept_len, scratch, scratch_bytes, batch,
                         draft_stride, P, vocab, stream=None):
    _check(load().dspark_greedy_accept(_ptr(logits), _ptr(draft), _ptr(proposal_len), _ptr(accepted),
                                       _ptr(accept_len), _ptr(scratch), scratch_bytes, batch, draft_stride, P,
                                       vocab, _stream(stream)), "dspark_greedy_accept")


def dspark_greedy_accept_noalloc(logits, draft, proposal_len, accepted, accept_len, batch, draft_stride, P, vocab,
                                 stream=None):
    """dspark_greedy_accept on the library's fixed scratch array (no device
    allocation by the library or by this wrapper); batch * (P + 1) must not
    exceed NOALLOC_MAX_VERIFY_ROWS.  Calls must not overlap on the GPU."""
    _check(load().dspark_greedy_accept_noalloc(_ptr(logits), _ptr(draft), _ptr(proposal_len), _ptr(accepted),
                                               _ptr(accept_len), batch, draft_stride, P, vocab, _stream(stream)),
           "dspark_greedy_accept_noalloc")


def dspark_check_noise_range(h0, L, n, stream=None):
    _check(load().dspark_check_noise_range(h0 & 0xFFFFFFFF, _ptr(L), n, _stream(stream)), "dspark_check_noise_range")


def dspark_check_hash(seed, step, pos, salt, ids, out, n, stream=None):
    _check(load().dspark_check_hash(seed, step, pos, salt & 0xFFFFFFFF, _ptr(ids), _ptr(out), n, _stream(stream)),
           "dspark_check_hash")


def dspark_check_logit(base, bias, c, l, n, mult, cap, stream=None):
    _check(load().dspark_check_logit(_ptr(base), _ptr(bias), _ptr(c), _ptr(l), n, mult, cap, _stream(stream)),
           "dspark_check_logit")


def dspark_check_key(l, temp, h, key, n, stream=None):
    _check(load().dspark_check_key(_ptr(l), temp, _ptr(h), _ptr(key), n, _stream(stream)), "dspark_check_key")


def dspark_check_logf(x, y, n, stream=None):
    _check(load().dspark_check_logf(_ptr(x), _ptr(y), n, _stream(stream)), "dspark_check_logf")


def dspark_check_tanhf(x, y, n, stream=None):
    _check(load().dspark_check_tanhf(_ptr(x), _ptr(y), n, _stream(stream)), "dspark_check_tanhf")


def dspark_check_expf(x, y, n, stream=None):
    _check(load().dspark_check_expf(_ptr(x), _ptr(y), n, _stream(stream)), "dspark_check_expf")


def dspark_check_div(x, d, y, n, stream=None):
    _check(load().dspark_check_div(_ptr(x), d, _ptr(y), n, _stream(stream)), "dspark_check_div")


def dspark_check_div_sweep(d, lo, n, out, stream=None):
    _check(load().dspark_check_div_sweep(d, lo, n, _ptr(out), _stream(stream)), "dspark_check_div_sweep")


def dspark_fill_uniforms(uniforms, n, seed, offset, stream=None):
    _check(load().dspark_fill_uniforms(_ptr(uniforms), n, seed & (2**64 - 1), offset & (2**64 - 1),
                                       _stream(stream)), "dspark_fill_uniforms")


def dspark_probabilistic_accept(target_probs, draft_probs, draft, proposal_len, uniforms, accepted, accept_len,
                                batch, draft_stride, P, vocab, stream=None):
    _check(load().dspark_probabilistic_accept(_ptr(target_probs), _ptr(draft_probs), _ptr(draft),
                                              _ptr(proposal_len), _ptr(uniforms), _ptr(accepted),
                                              _ptr(accept_len), batch, draft_stride, P, vocab, _stream(stream)),
           "dspark_probabilistic_accept")


def dspark_logits_to_probs(logits, probs, rows, vocab, temperature, top_k, top_p, stream=None):
    _check(load().dspark_logits_to_probs(_ptr(logits), _ptr(probs), rows, vocab, temperature, top_k, top_p,
                                         _stream(stream)), "dspark_logits_to_probs")


def dspark_quantize_w2_fp8(w2_bf16, w2_fp8, scale_f16, vocab, rank, stream=None):
    _check(load().dspark_quantize_w2_fp8(_ptr(w2_bf16), _ptr(w2_fp8), _ptr(scale_f16), vocab, rank, _stream(stream)),
           "dspark_quantize_w2_fp8")


def dspark_noise_bound_tables(n: int = 512):
    """The step kernel's noise bounds (host code): (ub, lb) float32 arrays."""
    ub = (ctypes.c_float * n)()
    lb = (ctypes.c_float * n)()
    rc = load().dspark_noise_bound_tables(ub, lb, n)
    if rc < 0:
        _check(rc, "dspark_noise_bound_tables")
    return list(ub)[:rc], list(lb)[:rc]


# --------------------------------------------------------------------------
# The paged 4-bit key/value cache (include/dspark_kv4.h)
# --------------------------------------------------------------------------

_dtypes: dict = {}


def _dtype(t) -> int:
    if not _dtypes:
        import torch
        _dtypes.update({torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32})
    code = _dtypes.get(t.dtype)
    if code is None:
        raise TypeError(f"bfloat16, float16 or float32 tensors are wanted: got {t.dtype}")
    return code


_int32 = None


def _want_int32(**tensors):
    global _int32
    if _int32 is None:
        import torch
        _int32 = torch.int32
    for name, t in tensors.items():
        if t is not None and (t.dtype is not _int32 or not t.is_contiguous()):
            raise TypeError(f"{name}: a contiguous int32 tensor is wanted")


def _want_table(name, t, slots):
    """Rows of page ids, one for each slot."""
    if t.dim() != 2 or t.dtype is not _int32 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise TypeError(f"{name}: int32 [slots, pages] with contiguous pages is wanted")
    if t.shape[0] < slots:
        raise ValueError(f"{name}: a row for each of lens' slots is wanted")


def _rows3(name, t):
    """Pointer and element strides of a [rows, heads, dim] tensor."""
    if t is None:
        return None, 0, 0
    strides = t.stride()
    if len(strides) != 3 or strides[2] != 1:
        raise ValueError(f"{name}: [rows, heads, dim] with contiguous dim is wanted")
    return t.data_ptr(), strides[0], strides[1]


def kv4_page_bytes(page_size: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of a page: what data's rows of Kv4Cache hold."""
    return kv_heads * page_size * (head_dim + head_dim // 8)


class Kv4Cache:
    """One layer's cache: data uint8 [num_pages, page bytes] (device; a row
    stride larger than the page's bytes is allowed), scales FP32 [kv_heads]
    or None."""

    def __init__(self, data, page_size, kv_heads, head_dim, *, k_scale=None, v_scale=None):
        import torch
        if data.dim() != 2 or data.dtype != torch.uint8 or data.stride(1) != 1:
            raise ValueError("data: uint8 [num_pages, page bytes] with contiguous bytes is wanted")
        if data.shape[1] < kv4_page_bytes(page_size, kv_heads, head_dim):
            raise ValueError("data: a page holds fewer bytes than its records")
        for s in (k_scale, v_scale):
            if s is not None and (s.dtype != torch.float32 or s.numel() != kv_heads or not s.is_contiguous()):
                raise ValueError("scales: contiguous float32 [kv_heads] is wanted")
        self.data, self.k_scale, self.v_scale = data, k_scale, v_scale  # keep them alive
        self.head_dim, self.kv_heads = head_dim, kv_heads
        self.struct = Kv4CacheStruct(_ptr(data), data.stride(0), data.shape[0], page_size, kv_heads, head_dim,
                                     _ptr(k_scale), _ptr(v_scale))
        self.ref = ctypes.addressof(self.struct)


class Kv4Batch:
    """The requests of a step: row_start int32 [batch + 1], lens int32
    [max_slots], table int32 [max_slots, pages], slots int32 [batch] or None
    (request i in slot i)."""

    def __init__(self, row_start, lens, table, *, total_rows, max_rows, slots=None):
        _want_int32(row_start=row_start, lens=lens, slots=slots)
        _want_table("table", table, lens.numel())
        if slots is not None and slots.numel() != row_start.numel() - 1:
            raise ValueError("slots: one for each request is wanted")
        self.tensors = (row_start, lens, table, slots)  # keep them alive
        self.total_rows = total_rows
        self.struct = Kv4BatchStruct(row_start.numel() - 1, total_rows, max_rows, table.shape[1], lens.numel(), 0,
                                     _ptr(row_start), _ptr(slots), _ptr(lens), _ptr(table), table.stride(0))
        self.ref = ctypes.addressof(self.struct)


def _check_rows(cache, batch, heads, **tensors):
    for name, t in tensors.items():
        if t is None:
            continue
        rows, h, dim = t.shape
        if rows < batch.total_rows or h != heads or dim != cache.head_dim:
            raise ValueError(f"{name}: [total_rows, {heads}, {cache.head_dim}] is wanted: got {tuple(t.shape)}")


def dspark_kv4_append(cache: Kv4Cache, batch: Kv4Batch, k, v, stream=None):
    """Store the rows' keys and values [rows, kv_heads, head_dim]."""
    _check_rows(cache, batch, cache.kv_heads, k=k, v=v)
    if k.dtype != v.dtype:
        raise TypeError("k and v of one type are wanted")
    _check(load().dspark_kv4_append(cache.ref, batch.ref, *_rows3("k", k), *_rows3("v", v), _dtype(k),
                                    _stream(stream)), "dspark_kv4_append")


def dspark_kv4_read(cache: Kv4Cache, batch: Kv4Batch, k, v, stream=None):
    """The rows' cached keys and values into k, v (one of them may be None)."""
    _check_rows(cache, batch, cache.kv_heads, k=k, v=v)
    if k is not None and v is not None and k.dtype != v.dtype:
        raise TypeError("k and v of one type are wanted")
    _check(load().dspark_kv4_read(cache.ref, batch.ref, *_rows3("k", k), *_rows3("v", v),
                                  _dtype(v if k is None else k), _stream(stream)), "dspark_kv4_read")


def dspark_kv4_attention_workspace_bytes(cache: Kv4Cache, batch: Kv4Batch, q_heads: int) -> int:
    return int(load().dspark_kv4_attention_workspace_bytes(cache.ref, batch.ref, q_heads))


def dspark_kv4_attention(cache: Kv4Cache, batch: Kv4Batch, q, out, scale: float, workspace, *, window: int = 0,
                         lse=None, stream=None):
    """Attention of q [rows, q_heads, head_dim] over the cache into out; lse
    (FP32 [rows, q_heads], contiguous) gets the log of the sums of weights."""
    _check_rows(cache, batch, q.shape[1], q=q, out=out)
    if q.dtype != out.dtype:
        raise TypeError("q and out of one type are wanted")
    if lse is not None and (lse.dim() != 2 or lse.shape[0] < batch.total_rows or lse.shape[1] != q.shape[1]
                            or not lse.is_contiguous() or _dtype(lse) != DTYPE_F32):
        raise ValueError("lse: contiguous float32 [total_rows, q_heads] is wanted")
    a = Kv4AttentionArgs(*_rows3("q", q), *_rows3("out", out), _ptr(lse), q.shape[1], _dtype(q), scale, window,
                         workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _check(load().dspark_kv4_attention(cache.ref, batch.ref, ctypes.addressof(a), _stream(stream)),
           "dspark_kv4_attention")


class PagePool:
    """The pages of a cache: refs int32 [num_pages], table int32 [max_slots,
    pages], lens int32 [max_slots] (device)."""

    def __init__(self, refs, table, lens, page_size):
        _want_int32(refs=refs, lens=lens)
        _want_table("table", table, lens.numel())
        self.refs, self.table, self.lens = refs, table, lens  # keep them alive
        self.struct = PagePoolStruct(refs.numel(), page_size, lens.numel(), table.shape[1], _ptr(refs), _ptr(table),
                                     table.stride(0), _ptr(lens))
        self.ref = ctypes.addressof(self.struct)


def _want_list(first, *others):
    """int32 lists, the others at least as long as the first; its length."""
    n = first.numel()
    for t in (first, *others):
        if t.dtype is not _int32 or not t.is_contiguous():
            raise TypeError("contiguous int32 tensors are wanted")
        if t.numel() < n:
            raise ValueError("lists: one entry for each slot is wanted")
    return n


def dspark_pages_trim(pool: PagePool, slots, new_len, stream=None):
    """Cut the slots back to new_len tokens (0 frees a slot)."""
    n = _want_list(slots, new_len)
    _check(load().dspark_pages_trim(pool.ref, n, slots.data_ptr(), new_len.data_ptr(), _stream(stream)),
           "dspark_pages_trim")


def dspark_pages_fork(pool: PagePool, src, dst, stream=None):
    """Make slots dst branches of slots src, on the same pages."""
    n = _want_list(src, dst)
    _check(load().dspark_pages_fork(pool.ref, n, src.data_ptr(), dst.data_ptr(), _stream(stream)),
           "dspark_pages_fork")


def dspark_pages_grow(pool: PagePool, slots, add, copy_src, copy_dst, granted, stream=None):
    """Room for add more tokens in each slot; pages to copy, and which slots
    got their room."""
    n = _want_list(slots, add, copy_src, copy_dst, granted)
    _check(load().dspark_pages_grow(pool.ref, n, slots.data_ptr(), add.data_ptr(), copy_src.data_ptr(),
                                    copy_dst.data_ptr(), granted.data_ptr(), _stream(stream)), "dspark_pages_grow")


def dspark_pages_compact(pool: PagePool, table_out, refs_out, map, move_src, move_dst, count, stream=None):
    """Move the live pages to the lowest ids: new tables and reference counts,
    and the moves of page data that they ask for."""
    _want_list(pool.refs, refs_out, map, move_src, move_dst)
    _want_int32(count=count)
    _want_table("table_out", table_out, 0)
    if table_out.shape != pool.table.shape or table_out.stride(0) != pool.table.stride(0):
        raise ValueError("table_out: the pool's table's shape and strides are wanted")
    _check(load().dspark_pages_compact(pool.ref, _ptr(table_out), _ptr(refs_out), _ptr(map), _ptr(move_src),
                                       _ptr(move_dst), _ptr(count), _stream(stream)), "dspark_pages_compact")


def dspark_pages_copy(data, src, dst, *, count=None, stream=None):
    """Copy pages src to dst in data, uint8 [num_pages, page bytes] or, for
    several layers, [layers, num_pages, page bytes]."""
    _want_int32(count=count)
    n = _want_list(src, dst)
    shape, strides = data.shape, data.stride()
    if len(shape) not in (2, 3) or strides[-1] != 1 or data.element_size() != 1:
        raise ValueError("data: bytes [num_pages, page bytes] or [layers, num_pages, page bytes] are wanted")
    layers, layer_stride = (1, 0) if len(shape) == 2 else (shape[0], strides[0])
    _check(load().dspark_pages_copy(data.data_ptr(), shape[-2], shape[-1], strides[-2], layers, layer_stride, n,
                                    src.data_ptr(), dst.data_ptr(), _ptr(count), _stream(stream)),
           "dspark_pages_copy")


# --------------------------------------------------------------------------
# torch convenience: one context over device tables, loop args from tensors
# --------------------------------------------------------------------------

def loop_args(*, base, cache, input_ids, anchor_idx, sample_pos, seeds, temperature, tokens, req_idx=None,
              mult=1.0, cap=0.0, salt=1 << 30, bias_out=None, rows=None, steps=None) -> LoopArgs:
    """LoopArgs from torch tensors (int16/bfloat16 storage for BF16)."""
    R = rows if rows is not None else base.shape[0]
    K = steps if steps is not None else base.shape[1]
    a = LoopArgs()
    a.rows, a.steps = R, K
    a.base, a.base_s0, a.base_s1 = _ptr(base), base.stride(0), base.stride(1)
    if cache is not None:
        a.cache, a.cache_s0, a.cache_s1 = _ptr(cache), cache.stride(0), cache.stride(1)
    a.input_ids, a.anchor_idx = _ptr(input_ids), _ptr(anchor_idx)
    if req_idx is not None:
        a.req_idx, a.req_s0 = _ptr(req_idx), req_idx.stride(0)
    a.sample_pos, a.pos_s0 = _ptr(sample_pos), sample_pos.stride(0)
    a.num_req = seeds.shape[0]
    a.seeds, a.temperature = _ptr(seeds), _ptr(temperature)
    a.mult, a.cap, a.salt = float(mult), float(cap), int(salt) & 0xFFFFFFFF
    a.tokens, a.tokens_s0 = _ptr(tokens), tokens.stride(0)
    a.bias_out = _ptr(bias_out)
    return a


class MarkovContext:
    """Owns one dspark_markov_ctx over device w1 / w2 tables."""

    def __init__(self, w1, w2, *, max_rows, max_steps, flags=FLAG_PDL, stream=None):
        self.w1, self.w2 = w1, w2  # keep the tables alive
        self.vocab = int(w2.shape[0])
        self.ctx = dspark_markov_init(self.vocab, int(w2.shape[1]), int(w1.shape[0]), max_rows, max_steps,
                                      flags, w1, w2, stream)

    def loop(self, args: LoopArgs, stream=None):
        dspark_markov_loop(self.ctx, args, stream)

    def anchor(self, args: LoopArgs, stream=None):
        dspark_markov_anchor(self.ctx, args, stream)

    def step(self, args: LoopArgs, step: int, stream=None):
        dspark_markov_step(self.ctx, args, step, stream)

    def shard_step(self, args: LoopArgs, step: int, vocab_offset: int, packets, stream=None):
        dspark_markov_shard_step(self.ctx, args, step, vocab_offset, packets, stream)

    def pick(self, packets, tp: int, rows: int, tokens, step: int, stream=None):
        dspark_markov_pick(self.ctx, packets, tp, rows, tokens, tokens.stride(0), step, stream)

    def partial_count(self) -> int:
        return dspark_markov_partial_count(self.ctx)

    def bias_path(self, rows: int) -> int:
        return dspark_markov_bias_path(self.ctx, rows)

    def loop_kernels(self, args: LoopArgs) -> int:
        return dspark_markov_loop_kernels(self.ctx, args)

    def set_w2_fp8(self, w2_fp8, w2_scale_f16) -> None:
        """Attach E4M3 w2 and FP16 row scales (device tensors the caller keeps
        alive); None, None detaches."""
        dspark_markov_set_w2_fp8(self.ctx, w2_fp8, w2_scale_f16)
        self._fp8 = (w2_fp8, w2_scale_f16)

    def status(self, stream=None) -> int:
        return dspark_markov_get_status(self.ctx, stream)

    def status_detail(self, stream=None) -> list:
        return dspark_markov_get_status_detail(self.ctx, stream)

    def close(self):
        if self.ctx:
            dspark_markov_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
