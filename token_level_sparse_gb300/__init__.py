"""Python binding of libtokenselect (token-level KV selection, sm_103a).

Argument marshalling only: every function below passes device pointers and
sizes to the C ABI declared in include/tokenselect.h, under the same names,
and raises TokenSelectError on a non-OK status. All arithmetic of the decode
step runs in the CUDA kernels of the library. There is no CPU fallback: if
libtokenselect.so is missing the import of the library fails loudly.

Tensors are torch tensors on the context's device; ``None`` passes NULL.
Streams default to torch's current stream.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_char_p, c_double, c_float, c_int, c_int64, c_void_p

__all__ = [
    "TokenSelectError", "Config", "SelectParams", "library", "library_path",
    "TS_KV_F32", "TS_KV_BF16", "TS_KV_Q4", "TS_SELECT_TOPK", "TS_SELECT_TOPP", "STATUS",
    "TS_SCORE_HEAD_SOFT_VOTE", "TS_SCORE_LOGIT_SUM", "TS_SCORE_HEAD_HARD_VOTE", "ts_score_fn",
    "ts_prefill_chunk", "ts_select_blocks", "ts_append_kv", "ts_append_prompt", "ts_read_kv", "ts_attend",
    "ts_prompt_attend", "ts_page_bytes", "RopeConfig", "Rope", "ROPE_SCALING", "ts_rope_create", "ts_rope_destroy",
    "ts_rope_read", "ts_rotate", "ts_append_rotated", "ts_tree_attend", "ts_verify_tree", "ts_keep_rows",
    "ts_create", "ts_destroy", "ts_cache_create", "ts_cache_destroy", "ts_cache_reset",
    "ts_cache_check", "ts_score", "ts_select", "ts_sparse_attend", "ts_decode_step",
    "ts_get_status", "ts_status_str", "ts_version", "ts_profile_enable", "ts_profile_read",
    "ts_kernel_count", "ts_debug_phase_ns", "ts_sparse_attend_noalloc", "ts_set_wait_limit",
    "ts_inject_barrier_skip", "Context", "Cache", "Profile", "PROF_FAMILIES",
]

TS_KV_F32, TS_KV_BF16, TS_KV_Q4 = 0, 1, 2
TS_SELECT_TOPK, TS_SELECT_TOPP = 0, 1
TS_SCORE_HEAD_SOFT_VOTE, TS_SCORE_LOGIT_SUM, TS_SCORE_HEAD_HARD_VOTE = 0, 1, 2
STATUS = {
    0: "TS_OK", 1: "TS_ERR_INVALID_ARG", 2: "TS_ERR_SHAPE", 3: "TS_ERR_UNSUPPORTED",
    4: "TS_ERR_CUDA", 5: "TS_ERR_PAGE_OOB", 6: "TS_ERR_CAPACITY", 7: "TS_ERR_TIMEOUT",
    8: "TS_ERR_COOP_UNAVAILABLE", 9: "TS_ERR_SEQ_LEN", 10: "TS_ERR_SCRATCH_LIMIT",
}
STATUS_CODE = {v: k for k, v in STATUS.items()}

library_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtokenselect.so")


class TokenSelectError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class Config(ctypes.Structure):
    _fields_ = [("n_q_heads", c_int), ("n_kv_heads", c_int), ("head_dim", c_int),
                ("page_size", c_int), ("kv_dtype", c_int), ("max_batch", c_int),
                ("max_pages_per_seq", c_int), ("num_pages", c_int64)]


ROPE_SCALING = {"plain": 0, "linear": 1, "base": 2, "bands": 3, "yarn": 4, "given": 5}


class RopeConfig(ctypes.Structure):
    _fields_ = [("rot_dim", c_int), ("interleaved", c_int), ("scaling", c_int), ("base", c_double), ("factor", c_double),
                ("original", c_int), ("low", c_double), ("high", c_double), ("attention", c_double),
                ("freqs", POINTER(c_double))]


class Profile(ctypes.Structure):
    _fields_ = [("ms", c_double * 6), ("launches", c_int64 * 6)]


PROF_FAMILIES = ("check", "score", "vote", "select", "attend", "step")


class SelectParams(ctypes.Structure):
    _fields_ = [("mode", c_int), ("k", c_int), ("n_sink", c_int), ("n_local", c_int),
                ("top_p", c_float), ("theta", c_float), ("softmax_scale", c_float), ("score_fn", c_int)]


_lib = None
_SIGS = {
    "ts_version": (c_int, []),
    "ts_status_str": (c_char_p, [c_int]),
    "ts_create": (c_int, [POINTER(c_void_p), POINTER(Config)]),
    "ts_destroy": (c_int, [c_void_p]),
    "ts_cache_create": (c_int, [c_void_p, POINTER(c_void_p), c_int, c_int]),
    "ts_cache_destroy": (c_int, [c_void_p]),
    "ts_cache_reset": (c_int, [c_void_p, c_void_p]),
    "ts_cache_check": (c_int, [c_void_p, c_void_p, c_int, c_void_p, c_int, c_float, c_void_p,
                               c_void_p, c_void_p]),
    "ts_score": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p,
                         c_float, c_void_p, c_int64, c_void_p]),
    "ts_score_fn": (c_int, [c_void_p, POINTER(SelectParams), c_void_p, c_void_p, c_void_p, c_void_p, c_int,
                            c_void_p, c_void_p, c_int64, c_void_p]),
    "ts_select": (c_int, [c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_int64, c_void_p, c_int,
                          c_void_p, POINTER(SelectParams), c_void_p, c_int64, c_void_p, c_void_p]),
    "ts_sparse_attend": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_int64, c_void_p, c_int, c_float, c_void_p, c_void_p, c_void_p]),
    "ts_decode_step": (c_int, [c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                               c_void_p, c_int, POINTER(SelectParams), c_void_p, c_int64, c_void_p,
                               c_int64, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "ts_get_status": (c_int, [c_void_p, POINTER(c_int), c_void_p]),
    "ts_append_kv": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_void_p]),
    "ts_select_blocks": (c_int, [c_void_p, c_void_p, c_int64, c_void_p, c_int, c_int, c_int, c_void_p, c_int64,
                                 c_void_p, c_void_p]),
    "ts_prefill_chunk": (c_int, [c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_int,
                                 POINTER(SelectParams), c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p,
                                 c_void_p, c_void_p]),
    "ts_append_prompt": (c_int, [c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p, c_int, c_int,
                                 c_void_p, c_void_p, c_void_p, c_void_p]),
    "ts_read_kv": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                           c_void_p, c_void_p]),
    "ts_attend": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_float, c_void_p,
                          c_void_p, c_void_p]),
    "ts_prompt_attend": (c_int, [c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int,
                                 c_int, c_float, c_void_p, c_int64, c_void_p, c_void_p]),
    "ts_page_bytes": (c_int64, [POINTER(Config)]),
    "ts_rope_create": (c_int, [POINTER(c_void_p), POINTER(RopeConfig)]),
    "ts_rope_destroy": (c_int, [c_void_p]),
    "ts_rope_read": (c_int, [c_void_p, POINTER(c_double), POINTER(c_double)]),
    "ts_rotate": (c_int, [c_void_p, c_void_p, c_void_p, c_int64, c_int, c_int, c_void_p, c_int, c_void_p, c_int64, c_int,
                          c_void_p]),
    "ts_append_rotated": (c_int, [c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p, c_void_p,
                                  c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_int,
                                  c_void_p]),
    "ts_tree_attend": (c_int, [c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                               c_int, c_int, c_int, c_float, c_void_p, c_int64, c_void_p, c_void_p]),
    "ts_verify_tree": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_void_p, c_int64, c_void_p,
                               c_int64, c_void_p, c_void_p, c_int, c_void_p, c_int64, c_void_p, c_void_p, c_void_p]),
    "ts_keep_rows": (c_int, [c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_int, c_int, c_void_p, c_void_p,
                             c_void_p, c_int, c_int64, c_void_p, c_void_p]),
    "ts_set_wait_limit": (c_int, [c_void_p, ctypes.c_uint64]),
    "ts_inject_barrier_skip": (c_int, [c_void_p, c_int, c_int]),
    "ts_profile_enable": (c_int, [c_void_p, c_int]),
    "ts_profile_read": (c_int, [c_void_p, c_void_p, c_int]),
    "ts_kernel_count": (c_int, [c_void_p, POINTER(c_int64)]),
    "ts_debug_phase_ns": (c_int, [c_void_p, c_void_p, c_void_p]),
    "ts_sparse_attend_noalloc": (c_int, [c_int, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p, c_int64,
                                         c_void_p, c_int, c_void_p, c_int64, c_void_p, c_int, c_float,
                                         c_void_p, c_void_p, c_void_p, c_void_p]),
}


def library() -> ctypes.CDLL:
    """The loaded libtokenselect.so (built in-tree by token_level_sparse_gb300.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise ImportError(f"{library_path} is missing: build it with "
                              "`python -m token_level_sparse_gb300.build` (nvcc, sm_103a)")
        lib = ctypes.CDLL(library_path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(st: int, where: str):
    if st != 0:
        raise TokenSelectError(st, where)


def _p(t):
    """Device pointer of a tensor (None -> NULL; ints pass through)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _packed(where, shapes, dtypes, on_device):
    """Refuses a packed call: shapes and dtypes are (got, wanted) pairs, on_device the tensors (None: absent)."""
    for got, want in shapes:
        if got != want:
            raise TokenSelectError(STATUS_CODE["TS_ERR_SHAPE"], f"{where}: {tuple(got)} instead of {tuple(want)}")
    for got, want in dtypes:
        if got is not want:
            raise TokenSelectError(STATUS_CODE["TS_ERR_INVALID_ARG"], f"{where}: {got} instead of {want}")
    for t in on_device:
        if t is not None and t.get_device() != _device():
            raise TokenSelectError(STATUS_CODE["TS_ERR_INVALID_ARG"], f"{where}: a tensor is not on the current device")


def _refuse(where, status, why):
    raise TokenSelectError(STATUS_CODE[status], f"{where}: {why}")


def _tensors(where, *specs):
    """Refuses a call unless every (tensor, elements, type) is dense, of this type, on the current device and holds as
    many elements or more. None and raw addresses are not looked at, here and below: the library sees to the first,
    nobody can to the second."""
    here = _device()
    for t, elements, dtype in specs:
        if t is None or isinstance(t, int):
            continue
        if t.dtype is dtype and t.numel() >= elements and t.is_contiguous() and t.get_device() == here:
            continue
        if t.numel() < elements:
            _refuse(where, "TS_ERR_SHAPE", f"{tuple(t.shape)}: less than {elements} elements")
        if t.dtype is not dtype:
            _refuse(where, "TS_ERR_INVALID_ARG", f"{t.dtype} instead of {dtype}")
        _refuse(where, "TS_ERR_INVALID_ARG", "a tensor is not dense or not on the current device")


def _rows_of(where, B, *specs):
    """The same for (tensor, type) with a row for each sequence, rows dense in themselves."""
    here = _device()
    for t, dtype in specs:
        if t is None or isinstance(t, int):
            continue
        if t.dim() != 2 or t.shape[0] < B:
            _refuse(where, "TS_ERR_SHAPE", f"{tuple(t.shape)} instead of {B} rows")
        if t.dtype is not dtype:
            _refuse(where, "TS_ERR_INVALID_ARG", f"{t.dtype} instead of {dtype}")
        if t.stride(1) != 1 or t.get_device() != here:
            _refuse(where, "TS_ERR_INVALID_ARG", "a tensor's rows are not dense, or not on the current device")


def _dense(where, *tensors):
    for t in tensors:
        if t is not None and not t.is_contiguous():
            raise TokenSelectError(STATUS_CODE["TS_ERR_INVALID_ARG"], f"{where}: a tensor is not dense")


def _row_stride(t, total, row):
    """Elements from row to row of a packed [total][heads][d] tensor, which must be dense inside a row."""
    heads, d = row
    rows, head, one = t.stride()        # (one call: each takes as long as all three)
    if (one != 1 and d > 1) or (head != d and heads > 1):
        raise TokenSelectError(STATUS_CODE["TS_ERR_INVALID_ARG"], "a packed row is not dense")
    return rows if total > 1 else heads * d


_stream_of = _device = _bfloat16 = _float32 = _int32 = None


def _torch():
    """What the calls below need of torch, looked up at the first call that needs it (raw calls with raw streams
    need none of it)."""
    global _stream_of, _device, _bfloat16, _float32, _int32
    import torch
    _bfloat16, _float32, _int32 = torch.bfloat16, torch.float32, torch.int32
    _device = torch.cuda.current_device
    _stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if _stream_of is None:
        _stream_of = lambda device: torch.cuda.current_stream(device).cuda_stream


def _current_stream():
    """The raw handle of torch's current stream (without the Stream object, whose making takes microseconds)."""
    if _device is None:
        _torch()
    return _stream_of(_device())


def _s(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _params(mode=TS_SELECT_TOPK, k=2048, n_sink=4, n_local=512, top_p=0.9, theta=0.9, softmax_scale=0.0,
            score_fn=TS_SCORE_HEAD_SOFT_VOTE):
    if isinstance(mode, SelectParams):
        return mode
    return SelectParams(mode, k, n_sink, n_local, top_p, theta, softmax_scale, score_fn)


# ---------------------------------------------------------------- raw calls

def ts_version() -> int:
    return library().ts_version()


def ts_status_str(status: int) -> str:
    return library().ts_status_str(status).decode()


def ts_create(cfg: Config) -> int:
    h = c_void_p()
    _check(library().ts_create(ctypes.byref(h), ctypes.byref(cfg)), "ts_create")
    return h.value


def ts_destroy(ctx: int) -> None:
    _check(library().ts_destroy(ctx), "ts_destroy")


def ts_cache_create(ctx: int, n_layers: int, capacity: int) -> int:
    h = c_void_p()
    _check(library().ts_cache_create(ctx, ctypes.byref(h), n_layers, capacity), "ts_cache_create")
    return h.value


def ts_cache_destroy(cache: int) -> None:
    _check(library().ts_cache_destroy(cache), "ts_cache_destroy")


def ts_cache_reset(cache: int, stream=None) -> None:
    _check(library().ts_cache_reset(cache, _s(stream)), "ts_cache_reset")


def ts_cache_check(ctx, cache, layer, q, B, theta, hit, cos_out=None, stream=None) -> None:
    _check(library().ts_cache_check(ctx, cache, layer, _p(q), B, theta, _p(hit), _p(cos_out), _s(stream)),
           "ts_cache_check")


def ts_score(ctx, q, k_pool, page_table, seq_lens, B, skip, scale, vote, vote_stride, stream=None) -> None:
    _check(library().ts_score(ctx, _p(q), _p(k_pool), _p(page_table), _p(seq_lens), B, _p(skip), scale,
                              _p(vote), vote_stride, _s(stream)), "ts_score")


def ts_score_fn(ctx, params, q, k_pool, page_table, seq_lens, B, skip, vote, vote_stride, stream=None) -> None:
    _check(library().ts_score_fn(ctx, ctypes.byref(params), _p(q), _p(k_pool), _p(page_table), _p(seq_lens), B,
                                 _p(skip), _p(vote), vote_stride, _s(stream)), "ts_score_fn")


def ts_select(ctx, cache, layer, q, vote, vote_stride, seq_lens, B, hit, params, idx, idx_stride, count,
              stream=None) -> None:
    _check(library().ts_select(ctx, cache, layer, _p(q), _p(vote), vote_stride, _p(seq_lens), B, _p(hit),
                               ctypes.byref(params), _p(idx), idx_stride, _p(count), _s(stream)), "ts_select")


def ts_sparse_attend(ctx, q, k_pool, v_pool, page_table, idx, idx_stride, count, B, scale, out, lse=None,
                     stream=None) -> None:
    _check(library().ts_sparse_attend(ctx, _p(q), _p(k_pool), _p(v_pool), _p(page_table), _p(idx),
                                      idx_stride, _p(count), B, scale, _p(out), _p(lse), _s(stream)),
           "ts_sparse_attend")


def ts_decode_step(ctx, cache, layer, q, k_pool, v_pool, page_table, seq_lens, B, params, vote, vote_stride,
                   idx, idx_stride, count, out, lse=None, hit=None, stream=None) -> None:
    _check(library().ts_decode_step(ctx, cache, layer, _p(q), _p(k_pool), _p(v_pool), _p(page_table),
                                    _p(seq_lens), B, ctypes.byref(params), _p(vote), vote_stride, _p(idx),
                                    idx_stride, _p(count), _p(out), _p(lse), _p(hit), _s(stream)),
           "ts_decode_step")


def ts_sparse_attend_noalloc(n_q_heads, n_kv_heads, head_dim, kv_dtype, q, k_pool, v_pool, num_pages,
                             page_table, max_pages_per_seq, idx, idx_stride, count, B, scale, out, lse=None,
                             status=None, stream=None) -> None:
    """Sparse attention with no context and no allocation (fixed static scratch)."""
    _check(library().ts_sparse_attend_noalloc(n_q_heads, n_kv_heads, head_dim, kv_dtype, _p(q), _p(k_pool),
                                              _p(v_pool), num_pages, _p(page_table), max_pages_per_seq, _p(idx),
                                              idx_stride, _p(count), B, scale, _p(out), _p(lse), _p(status),
                                              _s(stream)), "ts_sparse_attend_noalloc")


def ts_get_status(ctx, stream=None) -> int:
    v = c_int(0)
    _check(library().ts_get_status(ctx, ctypes.byref(v), _s(stream)), "ts_get_status")
    return v.value


def ts_prefill_chunk(ctx, q, c, k_pool, v_pool, page_table, seq_lens, B, params, vote, vote_stride, idx,
                     idx_stride, count, out, lse=None, stream=None) -> None:
    _check(library().ts_prefill_chunk(ctx, _p(q), c, _p(k_pool), _p(v_pool), _p(page_table), _p(seq_lens), B,
                                      ctypes.byref(params), _p(vote), vote_stride, _p(idx), idx_stride, _p(count),
                                      _p(out), _p(lse), _s(stream)), "ts_prefill_chunk")


def ts_select_blocks(ctx, vote, vote_stride, seq_lens, B, block, budget, idx, idx_stride, count, stream=None):
    _check(library().ts_select_blocks(ctx, _p(vote), vote_stride, _p(seq_lens), B, block, budget, _p(idx),
                                      idx_stride, _p(count), _s(stream)), "ts_select_blocks")


def ts_append_kv(ctx, k_new, v_new, page_table, seq_lens, B, k_pool, v_pool, stream=None) -> None:
    _check(library().ts_append_kv(ctx, _p(k_new), _p(v_new), _p(page_table), _p(seq_lens), B, _p(k_pool),
                                  _p(v_pool), _s(stream)), "ts_append_kv")


def ts_append_prompt(ctx, k, k_stride, v, v_stride, cu_rows, starts, B, total, page_table, k_pool, v_pool,
                     stream=None) -> None:
    _check(library().ts_append_prompt(ctx, _p(k), k_stride, _p(v), v_stride, _p(cu_rows), _p(starts), B, total,
                                      _p(page_table), _p(k_pool), _p(v_pool), _s(stream)), "ts_append_prompt")


def ts_read_kv(ctx, cu_rows, starts, B, total, page_table, k_pool, v_pool, k_out, v_out, stream=None) -> None:
    _check(library().ts_read_kv(ctx, _p(cu_rows), _p(starts), B, total, _p(page_table), _p(k_pool), _p(v_pool),
                                _p(k_out), _p(v_out), _s(stream)), "ts_read_kv")


def ts_attend(ctx, q, k_pool, v_pool, page_table, seq_lens, B, scale, out, lse=None, stream=None) -> None:
    _check(library().ts_attend(ctx, _p(q), _p(k_pool), _p(v_pool), _p(page_table), _p(seq_lens), B, scale, _p(out),
                               _p(lse), _s(stream)), "ts_attend")


def ts_prompt_attend(ctx, q, q_stride, k, k_stride, v, v_stride, cu_rows, B, total, scale, out, out_stride, lse=None,
                     stream=None) -> None:
    _check(library().ts_prompt_attend(ctx, _p(q), q_stride, _p(k), k_stride, _p(v), v_stride, _p(cu_rows), B, total,
                                      scale, _p(out), out_stride, _p(lse), _s(stream)), "ts_prompt_attend")


def ts_rope_create(cfg: RopeConfig) -> int:
    h = c_void_p()
    _check(library().ts_rope_create(ctypes.byref(h), ctypes.byref(cfg)), "ts_rope_create")
    return h.value


def ts_rope_destroy(rope: int) -> None:
    _check(library().ts_rope_destroy(rope), "ts_rope_destroy")


def ts_rope_read(rope: int, pairs: int):
    """(frequencies of the pairs in radians per position, factor of what is turned)."""
    f, a = (c_double * pairs)(), c_double()
    _check(library().ts_rope_read(rope, f, ctypes.byref(a)), "ts_rope_read")
    return list(f), a.value


def ts_rotate(ctx, rope, x, x_stride, dtype, heads, positions, total, out, out_stride, out_dtype, stream=None) -> None:
    _check(library().ts_rotate(ctx, rope, _p(x), x_stride, dtype, heads, _p(positions), total, _p(out), out_stride,
                               out_dtype, _s(stream)), "ts_rotate")


def ts_append_rotated(ctx, rope, k, k_stride, v, v_stride, positions, cu_rows, starts, B, total, page_table, k_pool,
                      v_pool, q=None, q_stride=0, q_out=None, q_out_stride=0, q_out_dtype=0, stream=None) -> None:
    _check(library().ts_append_rotated(ctx, rope, _p(k), k_stride, _p(v), v_stride, _p(positions), _p(cu_rows), _p(starts),
                                       B, total, _p(page_table), _p(k_pool), _p(v_pool), _p(q), q_stride, _p(q_out),
                                       q_out_stride, q_out_dtype, _s(stream)), "ts_append_rotated")


def ts_tree_attend(ctx, q, q_stride, k_pool, v_pool, page_table, seq_lens, cu_rows, mask, mask_words, B, total, scale, out,
                   out_stride, lse=None, stream=None) -> None:
    _check(library().ts_tree_attend(ctx, _p(q), q_stride, _p(k_pool), _p(v_pool), _p(page_table), _p(seq_lens), _p(cu_rows),
                                    _p(mask), mask_words, B, total, scale, _p(out), out_stride, _p(lse), _s(stream)),
           "ts_tree_attend")


def ts_verify_tree(ctx, tokens, parents, cu_rows, B, total, vocab, target, target_stride, draft, draft_stride, u, u_next,
                   distinct, path, path_stride, count, next_token, stream=None) -> None:
    _check(library().ts_verify_tree(ctx, _p(tokens), _p(parents), _p(cu_rows), B, total, vocab, _p(target), target_stride,
                                    _p(draft), draft_stride, _p(u), _p(u_next), distinct, _p(path), path_stride, _p(count),
                                    _p(next_token), _s(stream)), "ts_verify_tree")


def ts_keep_rows(ctx, path, path_stride, count, cu_rows, seq_lens, B, total, page_table, k_pool, v_pool, n_layers=1,
                 layer_bytes=0, new_lens=None, stream=None) -> None:
    _check(library().ts_keep_rows(ctx, _p(path), path_stride, _p(count), _p(cu_rows), _p(seq_lens), B, total,
                                  _p(page_table), _p(k_pool), _p(v_pool), n_layers, layer_bytes, _p(new_lens),
                                  _s(stream)), "ts_keep_rows")


def ts_page_bytes(cfg: Config) -> int:
    """Bytes of one page of a K pool (or a V pool), all KV heads."""
    return library().ts_page_bytes(ctypes.byref(cfg))


def ts_set_wait_limit(ctx, ns: int) -> None:
    _check(library().ts_set_wait_limit(ctx, int(ns)), "ts_set_wait_limit")


def ts_inject_barrier_skip(ctx, cta: int, barrier: int) -> None:
    _check(library().ts_inject_barrier_skip(ctx, cta, barrier), "ts_inject_barrier_skip")


def ts_profile_enable(ctx, on: bool) -> None:
    _check(library().ts_profile_enable(ctx, 1 if on else 0), "ts_profile_enable")


def ts_profile_read(ctx, keep: bool = False) -> dict:
    """{family: (ms, launches)} added up over the recorded brackets."""
    p = Profile()
    _check(library().ts_profile_read(ctx, ctypes.byref(p), 1 if keep else 0), "ts_profile_read")
    return {f: (p.ms[i], p.launches[i]) for i, f in enumerate(PROF_FAMILIES)}


def ts_debug_phase_ns(ctx, stream=None) -> list:
    """Phase-boundary times (ns) of CTA 0 in the last persistent step kernel."""
    buf = (ctypes.c_uint64 * 64)()
    _check(library().ts_debug_phase_ns(ctx, buf, _s(stream)), "ts_debug_phase_ns")
    return list(buf)


def ts_kernel_count(ctx) -> int:
    v = c_int64(0)
    _check(library().ts_kernel_count(ctx, ctypes.byref(v)), "ts_kernel_count")
    return v.value


# ------------------------------------------------------- handle wrappers

class Context:
    """Owns a ts_ctx for one head geometry and pool; tensors in, nothing computed here."""

    def __init__(self, n_q_heads, n_kv_heads, head_dim, kv_dtype, max_batch, max_pages_per_seq,
                 num_pages, page_size=16):
        self.cfg = Config(n_q_heads, n_kv_heads, head_dim, page_size, kv_dtype, max_batch,
                          max_pages_per_seq, num_pages)
        self.handle = ts_create(self.cfg)
        self.max_tokens = max_pages_per_seq * page_size
        self.cfg_d = head_dim
        # what the packed calls compare their tensors with
        self._q_row, self._kv_row = (n_q_heads, head_dim), (n_kv_heads, head_dim)
        self._q4, self._f32 = kv_dtype == TS_KV_Q4, kv_dtype == TS_KV_F32
        self._pool_bytes, self._columns = num_pages * ts_page_bytes(self.cfg), max_pages_per_seq

    def _rows_dtype(self):
        """Element type of the rows that go into the pools."""
        return _float32 if self._f32 else _bfloat16

    def _paged(self, where, B, page_table, k_pool, v_pool):
        """Refuses a page table or pools smaller than the context's."""
        here, need = _device(), self._pool_bytes
        try:
            rows, columns = page_table.shape                       # (one test of all, as most calls pass it)
            if (columns == self._columns and rows >= B and page_table.dtype is _int32 and page_table.is_contiguous()
                    and k_pool.nbytes >= need and v_pool.nbytes >= need and k_pool.is_contiguous() and v_pool.is_contiguous()
                    and page_table.get_device() == here and k_pool.get_device() == here and v_pool.get_device() == here):
                return
        except (AttributeError, TypeError, ValueError):            # None, raw addresses, other shapes
            pass
        if page_table is not None and not isinstance(page_table, int):
            if page_table.dim() != 2 or page_table.shape[1] != self._columns:
                _refuse(where, "TS_ERR_SHAPE", f"{tuple(page_table.shape)} instead of {(B, self._columns)}")
            _tensors(where, (page_table, B * self._columns, _int32))
        for t in (k_pool, v_pool):
            if t is None or isinstance(t, int):
                continue
            if t.nbytes < need:
                _refuse(where, "TS_ERR_SHAPE", f"a pool of less than {need} bytes")
            if t.get_device() != here or not t.is_contiguous():
                _refuse(where, "TS_ERR_INVALID_ARG", "a pool is not dense or not on the current device")

    def _queries(self, where, q, page_table, k_pool, v_pool, seq_lens=None, out=None, lse=None, vote=None, idx=None,
                 count=None, flags=None):
        """Refuses what a call over a 4-bit cache would read or write beyond, or take for another type."""
        if _device is None:
            _torch()
        B, here = q.shape[0], _device()
        n = B * self._q_row[0] * self._q_row[1]
        if q.numel() != n:
            _refuse(where, "TS_ERR_SHAPE", f"{tuple(q.shape)} instead of {(B, *self._q_row)}")
        _tensors(where, (q, n, _float32), (out, n, _float32), (seq_lens, B, _int32), (lse, B * self._q_row[0], _float32),
                 (count, B, _int32))
        self._paged(where, B, page_table, k_pool, k_pool if v_pool is None else v_pool)
        if vote is not None or idx is not None:
            _rows_of(where, B, (vote, _float32), (idx, _int32))
        if flags is not None and not isinstance(flags, int):
            if flags.numel() < B or flags.element_size() != 1:
                _refuse(where, "TS_ERR_SHAPE", f"{tuple(flags.shape)} of {flags.dtype} instead of {(B,)} bytes")
            if flags.get_device() != here or not flags.is_contiguous():
                _refuse(where, "TS_ERR_INVALID_ARG", "a tensor is not dense or not on the current device")

    def close(self):
        if self.handle:
            ts_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def cache(self, n_layers, capacity):
        return Cache(self, n_layers, capacity)

    def score(self, q, k_pool, page_table, seq_lens, vote, skip=None, scale=0.0, stream=None):
        if self._q4:
            self._queries("score", q, page_table, k_pool, None, seq_lens, vote=vote, flags=skip)
        ts_score(self.handle, q, k_pool, page_table, seq_lens, q.shape[0], skip, scale, vote,
                 vote.stride(0), stream)

    def score_fn(self, params, q, k_pool, page_table, seq_lens, vote, skip=None, stream=None):
        if self._q4:
            self._queries("score_fn", q, page_table, k_pool, None, seq_lens, vote=vote, flags=skip)
        ts_score_fn(self.handle, params, q, k_pool, page_table, seq_lens, q.shape[0], skip, vote, vote.stride(0),
                    stream)

    def select(self, vote, seq_lens, params, idx, count, cache=None, layer=0, q=None, hit=None, stream=None):
        ts_select(self.handle, cache.handle if cache else None, layer, q, vote, vote.stride(0), seq_lens,
                  seq_lens.shape[0], hit, params, idx, idx.stride(0), count, stream)

    def sparse_attend(self, q, k_pool, v_pool, page_table, idx, count, out, lse=None, scale=0.0, stream=None):
        if self._q4:
            self._queries("sparse_attend", q, page_table, k_pool, v_pool, out=out, lse=lse, idx=idx, count=count)
        ts_sparse_attend(self.handle, q, k_pool, v_pool, page_table, idx, idx.stride(0), count, q.shape[0],
                         scale, out, lse, stream)

    def decode_step(self, q, k_pool, v_pool, page_table, seq_lens, params, idx, count, out, lse=None,
                    hit=None, vote=None, cache=None, layer=0, stream=None):
        if self._q4:
            self._queries("decode_step", q, page_table, k_pool, v_pool, seq_lens, out, lse, vote, idx, count, hit)
        ts_decode_step(self.handle, cache.handle if cache else None, layer, q, k_pool, v_pool, page_table,
                       seq_lens, q.shape[0], params, vote, vote.stride(0) if vote is not None else 0, idx,
                       idx.stride(0), count, out, lse, hit, stream)

    def prefill_chunk(self, q, k_pool, v_pool, page_table, seq_lens, params, idx, count, out, lse=None, vote=None,
                      stream=None):
        """q [B][c][H][d]: one selection from the chunk's mean query, causal attention of every query."""
        ts_prefill_chunk(self.handle, q, q.shape[1], k_pool, v_pool, page_table, seq_lens, q.shape[0], params,
                         vote, vote.stride(0) if vote is not None else 0, idx, idx.stride(0), count, out, lse, stream)

    def append_kv(self, k_new, v_new, page_table, seq_lens, k_pool, v_pool, stream=None):
        """k_new / v_new [B][H_kv][d]: the current token's rows into position seq_lens[b] - 1."""
        if _device is None:
            _torch()
        B, kind, here = seq_lens.shape[0], self._rows_dtype(), _device()
        elements = B * self._kv_row[0] * self._kv_row[1]
        for t in (k_new, v_new):
            if t is None or isinstance(t, int):
                continue
            # (any view of the rows' bits goes into a pool that holds them as they are)
            if t.numel() < elements or (t.dtype is not kind and t.element_size() != kind.itemsize):
                _refuse("append_kv", "TS_ERR_SHAPE", f"{tuple(t.shape)} of {t.dtype} instead of {(B, *self._kv_row)} of {kind}")
            if (t.dtype is not kind and self._q4) or t.get_device() != here or not t.is_contiguous():
                _refuse("append_kv", "TS_ERR_INVALID_ARG", f"dense rows of {kind} on the current device are wanted")
        if self._q4:
            _tensors("append_kv", (seq_lens, B, _int32))
            self._paged("append_kv", B, page_table, k_pool, v_pool)
        ts_append_kv(self.handle, k_new, v_new, page_table, seq_lens, seq_lens.shape[0], k_pool, v_pool, stream)

    def append_prompt(self, k, v, cu_rows, page_table, k_pool, v_pool, starts=None, stream=None):
        """k / v [total][H_kv][d], packed: row r of sequence b to position starts[b] + r - cu_rows[b]."""
        if _device is None:
            _torch()
        ks, B, i32, kind, here = k.shape, cu_rows.shape[0] - 1, _int32, self._rows_dtype(), _device()
        if not (ks[1:] == self._kv_row and v.shape == ks and k.dtype is kind and v.dtype is kind and cu_rows.dtype is i32
                and k.get_device() == here and v.get_device() == here and cu_rows.get_device() == here):
            _packed("append_prompt", ((ks[1:], self._kv_row), (v.shape, ks)), ((k.dtype, kind), (v.dtype, kind), (cu_rows.dtype, i32)),
                    (k, v, cu_rows))
        if starts is not None and not (starts.shape == (B,) and starts.dtype is i32 and starts.get_device() == here):
            _packed("append_prompt", ((starts.shape, (B,)),), ((starts.dtype, i32),), (starts,))
        _dense("append_prompt", cu_rows, starts)
        self._paged("append_prompt", B, page_table, k_pool, v_pool)
        total, row = ks[0], self._kv_row
        ts_append_prompt(self.handle, k, _row_stride(k, total, row), v, _row_stride(v, total, row), cu_rows, starts, B, total,
                         page_table, k_pool, v_pool, stream)

    def read_kv(self, cu_rows, page_table, k_pool, v_pool, k_out, v_out, starts=None, stream=None):
        """k_out / v_out fp32 [total][H_kv][d]: the values of the rows that append_prompt would write."""
        if _device is None:
            _torch()
        ks, B, i32, f32, here = k_out.shape, cu_rows.shape[0] - 1, _int32, _float32, _device()
        if not (ks[1:] == self._kv_row and v_out.shape == ks and k_out.dtype is f32 and v_out.dtype is f32
                and cu_rows.dtype is i32 and k_out.get_device() == here and v_out.get_device() == here and cu_rows.get_device() == here):
            _packed("read_kv", ((ks[1:], self._kv_row), (v_out.shape, ks)),
                    ((k_out.dtype, f32), (v_out.dtype, f32), (cu_rows.dtype, i32)), (k_out, v_out, cu_rows))
        if starts is not None and not (starts.shape == (B,) and starts.dtype is i32 and starts.get_device() == here):
            _packed("read_kv", ((starts.shape, (B,)),), ((starts.dtype, i32),), (starts,))
        _dense("read_kv", k_out, v_out, cu_rows, starts)
        self._paged("read_kv", B, page_table, k_pool, v_pool)
        ts_read_kv(self.handle, cu_rows, starts, B, ks[0], page_table, k_pool, v_pool, k_out, v_out, stream)

    def attend(self, q, k_pool, v_pool, page_table, seq_lens, out, lse=None, scale=0.0, stream=None):
        """q [B][H][d] attends to every cached token of its sequence (4-bit pools)."""
        if self._q4:
            self._queries("attend", q, page_table, k_pool, v_pool, seq_lens, out, lse)
        ts_attend(self.handle, q, k_pool, v_pool, page_table, seq_lens, q.shape[0], scale, out, lse, stream)

    def prompt_attend(self, q, k, v, cu_rows, out, lse=None, scale=0.0, stream=None):
        """q / out [total][H][d], k / v [total][H_kv][d] (bf16, packed): causal attention of every sequence."""
        if _device is None:
            _torch()
        qs, ks, bf, i32, here = q.shape, k.shape, _bfloat16, _int32, _device()
        if not (qs[1:] == self._q_row and ks[1:] == self._kv_row and ks[0] == qs[0] and v.shape == ks and out.shape == qs
                and q.dtype is bf and k.dtype is bf and v.dtype is bf and out.dtype is bf and cu_rows.dtype is i32
                and q.get_device() == here and k.get_device() == here and v.get_device() == here and out.get_device() == here and cu_rows.get_device() == here):
            _packed("prompt_attend", ((qs[1:], self._q_row), (ks[1:], self._kv_row), (ks[:1], qs[:1]), (v.shape, ks), (out.shape, qs)),
                    ((q.dtype, bf), (k.dtype, bf), (v.dtype, bf), (out.dtype, bf), (cu_rows.dtype, i32)), (q, k, v, out, cu_rows))
        if lse is not None and not (lse.shape == qs[:2] and lse.dtype is _float32 and lse.get_device() == here):
            _packed("prompt_attend", ((lse.shape, qs[:2]),), ((lse.dtype, _float32),), (lse,))
        _dense("prompt_attend", cu_rows, lse)
        total, row = qs[0], self._kv_row
        ts_prompt_attend(self.handle, q, _row_stride(q, total, self._q_row), k, _row_stride(k, total, row), v,
                         _row_stride(v, total, row), cu_rows, cu_rows.shape[0] - 1, total, scale, out,
                         _row_stride(out, total, self._q_row), lse, stream)

    def rope(self, rot_dim=None, **kw):
        """A Rope for this context's heads (all of each head turned where rot_dim is not given)."""
        return Rope(self.cfg.head_dim if rot_dim is None else rot_dim, **kw)

    def _heads(self, where, x, heads, total, here):
        """Refuses a packed [total][heads][d] tensor of another shape, type or device; its row stride and type."""
        kind, shape = x.dtype, x.shape
        f32 = kind is _float32
        if len(shape) == 3 and (f32 or kind is _bfloat16) and x.get_device() == here:
            rows, h, d = shape
            if rows == total and h == heads and d == self.cfg_d:
                step, head, one = x.stride()                       # (the test that most calls pass)
                if one == 1 and head == d:
                    return (step if rows > 1 else h * d), TS_KV_F32 if f32 else TS_KV_BF16
                return _row_stride(x, total, (h, d)), TS_KV_F32 if f32 else TS_KV_BF16
        if len(shape) != 3 or tuple(shape) != (total, heads, self.cfg_d):
            _refuse(where, "TS_ERR_SHAPE", f"{tuple(shape)} instead of {(total, heads, self.cfg_d)}")
        if not f32 and kind is not _bfloat16:
            _refuse(where, "TS_ERR_INVALID_ARG", f"{kind} instead of bfloat16 or float32")
        _refuse(where, "TS_ERR_INVALID_ARG", "a tensor is not on the current device")

    @staticmethod
    def _counted(where, here, *specs):
        """Refuses every (tensor, shape, type) that is not dense, of exactly this shape and type, on the current device."""
        for t, shape, dtype in specs:
            if t is None or (t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == here):
                continue
            if t.shape != shape:
                _refuse(where, "TS_ERR_SHAPE", f"{tuple(t.shape)} instead of {tuple(shape)}")
            if t.dtype is not dtype:
                _refuse(where, "TS_ERR_INVALID_ARG", f"{t.dtype} instead of {dtype}")
            _refuse(where, "TS_ERR_INVALID_ARG", "a tensor is not dense or not on the current device")

    def rotate(self, rope, x, positions, out, stream=None):
        """x / out [total][heads][d] (bf16 or fp32 each): rows turned by positions int32 [total]. out may be x."""
        if _device is None:
            _torch()
        if x.dim() != 3:
            _refuse("rotate", "TS_ERR_SHAPE", f"{tuple(x.shape)} instead of (rows, heads, {self.cfg_d})")
        here, (total, heads, _) = _device(), x.shape
        xs, kind = self._heads("rotate", x, heads, total, here)
        os_, out_kind = self._heads("rotate", out, heads, total, here)
        self._counted("rotate", here, (positions, (total,), _int32))
        ts_rotate(self.handle, rope.handle, x, xs, kind, heads, positions, total, out, os_, out_kind, stream)

    def append_rotated(self, rope, k, v, positions, cu_rows, page_table, k_pool, v_pool, starts=None, q=None, q_out=None,
                       stream=None):
        """append_prompt with K turned by positions int32 [total]; q [total][H][d] of the rows' type into q_out too."""
        if _device is None:
            _torch()
        here, B, total, kind = _device(), cu_rows.shape[0] - 1, k.shape[0], self._rows_dtype()
        ks, _ = self._heads("append_rotated", k, self._kv_row[0], total, here)
        vs, _ = self._heads("append_rotated", v, self._kv_row[0], total, here)
        qs = os_ = out_kind = 0
        if (q is None) != (q_out is None):
            _refuse("append_rotated", "TS_ERR_INVALID_ARG", "q and q_out come together")
        if q is not None:
            qs, _ = self._heads("append_rotated", q, self._q_row[0], total, here)
            os_, out_kind = self._heads("append_rotated", q_out, self._q_row[0], total, here)
        for t in (k, v) if q is None else (k, v, q):
            if t.dtype is not kind:
                _refuse("append_rotated", "TS_ERR_INVALID_ARG", f"{t.dtype} instead of {kind}")
        self._counted("append_rotated", here, (positions, (total,), _int32), (cu_rows, (B + 1,), _int32), (starts, (B,), _int32))
        self._paged("append_rotated", B, page_table, k_pool, v_pool)
        ts_append_rotated(self.handle, rope.handle, k, ks, v, vs, positions, cu_rows, starts, B, total, page_table, k_pool,
                          v_pool, q, qs, q_out, os_, out_kind, stream)

    def tree_attend(self, q, k_pool, v_pool, page_table, seq_lens, cu_rows, mask, out, lse=None, scale=0.0, stream=None):
        """q / out [total][H][d] (bf16): the last cached tokens of each sequence, a tree of drafts, over its whole cache.
        mask int32 [total][words]: bit j of a row is set where it sees draft j; None: the drafts up to its own."""
        if _device is None:
            _torch()
        here, B, total, heads = _device(), cu_rows.shape[0] - 1, q.shape[0], self._q_row[0]
        qs, kind = self._heads("tree_attend", q, heads, total, here)
        os_, out_kind = self._heads("tree_attend", out, heads, total, here)
        if kind != TS_KV_BF16 or out_kind != TS_KV_BF16:
            _refuse("tree_attend", "TS_ERR_INVALID_ARG", "bfloat16 rows are wanted")
        self._counted("tree_attend", here, (seq_lens, (B,), _int32), (cu_rows, (B + 1,), _int32), (lse, (total, heads), _float32))
        words = 0
        if mask is not None:
            if mask.dim() != 2:
                _refuse("tree_attend", "TS_ERR_SHAPE", f"{tuple(mask.shape)} instead of {(total, 'words')}")
            words = mask.shape[1]
            self._counted("tree_attend", here, (mask, (total, words), _int32))
            if words == 0 and total > 0:                           # (its address is NULL, which stands for no mask)
                _refuse("tree_attend", "TS_ERR_SHAPE", "a mask without words")
        self._paged("tree_attend", B, page_table, k_pool, v_pool)
        ts_tree_attend(self.handle, q, qs, k_pool, v_pool, page_table, seq_lens, cu_rows, mask, words, B, total, scale, out,
                       os_, lse, stream)

    def verify_tree(self, tokens, parents, cu_rows, target, draft, u, u_next, path, count, next_token, distinct=False,
                    stream=None):
        """target / draft fp32 [total][vocab] (draft None: drafts without probabilities): path int32 [B][most], count and
        next_token int32 [B] receive the nodes that the target keeps and the token behind them."""
        if _device is None:
            _torch()
        here, B, total = _device(), cu_rows.shape[0] - 1, tokens.shape[0]
        if target.dim() != 2 or target.shape[0] != total or (draft is not None and draft.shape != target.shape):
            _refuse("verify_tree", "TS_ERR_SHAPE", f"{tuple(target.shape)} instead of {(total, 'vocab')}, for both")
        _rows_of("verify_tree", total, (target, _float32), (draft, _float32))
        if path.dim() != 2 or path.shape[0] != B:
            _refuse("verify_tree", "TS_ERR_SHAPE", f"{tuple(path.shape)} instead of {(B, 'most')}")
        self._counted("verify_tree", here, (tokens, (total,), _int32), (parents, (total,), _int32), (cu_rows, (B + 1,), _int32),
                      (u, (total,), _float32), (u_next, (B,), _float32), (path, path.shape, _int32), (count, (B,), _int32),
                      (next_token, (B,), _int32))
        vocab = target.shape[1]
        ts_verify_tree(self.handle, tokens, parents, cu_rows, B, total, vocab, target, target.stride(0) if total > 1 else vocab,
                       draft, 0 if draft is None else (draft.stride(0) if total > 1 else vocab), u, u_next,
                       1 if distinct else 0, path, path.shape[1], count, next_token, stream)

    def keep_rows(self, path, count, cu_rows, seq_lens, page_table, k_pool, v_pool, new_lens=None, total=None, stream=None):
        """The K and V rows of path's nodes to the front of the drafts'. Pools of one layer, or [layers][...] with a pool
        each. total: rows that cu_rows may end at (any, where it is not given)."""
        if _device is None:
            _torch()
        here, B = _device(), cu_rows.shape[0] - 1
        if path.dim() != 2 or path.shape[0] != B:
            _refuse("keep_rows", "TS_ERR_SHAPE", f"{tuple(path.shape)} instead of {(B, 'most')}")
        self._counted("keep_rows", here, (path, path.shape, _int32), (count, (B,), _int32), (cu_rows, (B + 1,), _int32),
                      (seq_lens, (B,), _int32), (new_lens, (B,), _int32))
        layers, step = 1, 0
        if k_pool.dim() == (4 if self._q4 else 5):                 # [layers][...], dense throughout
            layers = k_pool.shape[0]
            if layers == 0:
                return
            if k_pool.shape != v_pool.shape or k_pool.dtype is not v_pool.dtype or k_pool.nbytes < layers * self._pool_bytes:
                _refuse("keep_rows", "TS_ERR_SHAPE", f"pools of {layers} layers that differ, or of less than {self._pool_bytes} bytes each")
            step = k_pool.nbytes // layers
        self._paged("keep_rows", B, page_table, k_pool, v_pool)
        ts_keep_rows(self.handle, path, path.shape[1], count, cu_rows, seq_lens, B, (1 << 30) if total is None else total,
                     page_table, k_pool, v_pool, layers, step, new_lens, stream)

    def select_blocks(self, vote, seq_lens, block, budget, idx, count, stream=None):
        ts_select_blocks(self.handle, vote, vote.stride(0), seq_lens, seq_lens.shape[0], block, budget, idx,
                         idx.stride(0), count, stream)

    def status(self, stream=None) -> int:
        return ts_get_status(self.handle, stream)


class Rope:
    """Owns a ts_rope: the frequencies of rotary positions. scaling is one of ROPE_SCALING; freqs: radians per position of
    each pair, for "given"."""

    def __init__(self, rot_dim, base=10000.0, interleaved=False, scaling="plain", factor=1.0, original=0, low=0.0, high=0.0,
                 attention=0.0, freqs=None):
        self.handle = None
        if scaling not in ROPE_SCALING:
            _refuse("rope", "TS_ERR_INVALID_ARG", f"{scaling} is none of {', '.join(ROPE_SCALING)}")
        if freqs is not None and len(freqs) != rot_dim // 2:
            _refuse("rope", "TS_ERR_SHAPE", f"{len(freqs)} frequencies instead of {rot_dim // 2}")
        self.rot_dim = rot_dim
        given = None if freqs is None else (c_double * len(freqs))(*[float(f) for f in freqs])
        self.handle = ts_rope_create(RopeConfig(rot_dim, 1 if interleaved else 0, ROPE_SCALING[scaling], base, factor, original,
                                                low, high, attention, given))

    def read(self):
        """(frequencies of the pairs in radians per position, factor of what is turned)."""
        return ts_rope_read(self.handle, self.rot_dim // 2)

    def close(self):
        if self.handle:
            ts_rope_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Cache:
    """Owns a ts_cache (Selection Cache state: C_Q, C_T per sequence and layer)."""

    def __init__(self, ctx: Context, n_layers: int, capacity: int):
        self.ctx = ctx
        self.handle = ts_cache_create(ctx.handle, n_layers, capacity)

    def reset(self, stream=None):
        ts_cache_reset(self.handle, stream)

    def check(self, layer, q, theta, hit, cos_out=None, stream=None):
        ts_cache_check(self.ctx.handle, self.handle, layer, q, q.shape[0], theta, hit, cos_out, stream)

    def close(self):
        if self.handle:
            ts_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def params(**kw) -> SelectParams:
    """SelectParams with the paper's defaults (k 2048, 4 sinks, 512 local, theta 0.9)."""
    return _params(**kw)
