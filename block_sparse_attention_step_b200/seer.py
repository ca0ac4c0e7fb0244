"""ctypes binding of ``libseer.so`` (the C ABI in ``include/seer.h``).

Argument marshalling only: every function takes torch tensors (device memory
for the device arguments), checks dtype and contiguity (the paged-cache
operators also shapes against the dims), passes raw pointers
and the current CUDA stream, and raises ``SeerError`` on a non-zero status.
All computation happens in the library's kernels.  The library must have been
built (``python -m block_sparse_attention_step_b200.build``); there is no
fallback path, a missing library raises at first use.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libseer.so")

SEER_OK = 0
SEER_ERR_CUDA = 3
STATUS_NAMES = {0: "SEER_OK", 1: "SEER_ERR_INVALID_ARG", 2: "SEER_ERR_UNSUPPORTED",
                3: "SEER_ERR_CUDA", 4: "SEER_ERR_WORKSPACE"}
DEV_NONFINITE_SCORE = 1
DEV_BAD_INDEX = 2
DEV_BAD_PAGE = 4
DEV_K_CLAMPED = 8
DEV_TIMEOUT = 16
DEV_NONFINITE_KV = 32
DEV_BAD_TOKENS = 64
DEV_BAD_POSITION = 128

CACHE_BF16, CACHE_E4M3, CACHE_INT8 = 0, 1, 2
_CACHE_TYPES = {torch.bfloat16: CACHE_BF16, torch.float8_e4m3fn: CACHE_E4M3,
                torch.int8: CACHE_INT8}

EXPORTS = (
    "seer_version", "seer_status_string", "seer_last_cuda_error", "seer_dims_default",
    "seer_k_from_sparsity",
    "seer_k_from_budget", "seer_fill_k", "seer_default_splits", "seer_step_workspace_bytes",
    "seer_pool_keys", "seer_gate_scores", "seer_block_select", "seer_block_select_unified",
    "seer_sparse_decode",
    "seer_combine", "seer_decode_step", "seer_decode_step_host", "seer_host_ptr_mapped",
    "seer_decode_step_noalloc",
    "seer_decode_step_fused", "seer_step_workspace_init",
    "seer_prefill_k_max", "seer_prefill_workspace_bytes", "seer_prefill",
    "seer_prefill_attention",
    "seer_block_lse_elems", "seer_sparse_decode_mass", "seer_block_mass",
    "seer_rope_table", "seer_append_rope",
    "seer_sparse_decode_q8_splits", "seer_window_decode_splits", "seer_split_workspace_bytes",
    "seer_sparse_decode_q8", "seer_window_decode", "seer_window_prefill",
)
NOALLOC_SCRATCH_BYTES = 16 << 20


class SeerError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        detail = _lib().seer_status_string(status).decode()
        if status == SEER_ERR_CUDA:
            detail += ": " + _lib().seer_last_cuda_error().decode()
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)} ({detail})")


class seer_dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("stride_page", ctypes.c_int64),
                ("stride_token", ctypes.c_int64), ("stride_head", ctypes.c_int64)]


class seer_step_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("seqlens", ctypes.c_void_p),
                ("w_gate", ctypes.c_void_p), ("kbar", ctypes.c_void_p),
                ("k_per_seq", ctypes.c_void_p), ("update_kbar", ctypes.c_int32),
                ("force_newest", ctypes.c_int32), ("k_max", ctypes.c_int32),
                ("num_splits", ctypes.c_int32), ("gate_scale", ctypes.c_float),
                ("softmax_scale", ctypes.c_float), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("out", ctypes.c_void_p),
                ("lse_out", ctypes.c_void_p), ("dev_status", ctypes.c_void_p),
                ("block_lse", ctypes.c_void_p), ("block_mass", ctypes.c_void_p),
                ("unified_heads", ctypes.c_int32), ("k_new", ctypes.c_void_p),
                ("v_new", ctypes.c_void_p)]


class seer_prefill_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("seqlens", ctypes.c_void_p),
                ("w_gate", ctypes.c_void_p), ("kbar", ctypes.c_void_p),
                ("pool_keys", ctypes.c_int32), ("sparsity_permille", ctypes.c_int32),
                ("budget_tokens", ctypes.c_int32), ("k_max", ctypes.c_int32),
                ("gate_scale", ctypes.c_float), ("softmax_scale", ctypes.c_float),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("out", ctypes.c_void_p), ("lse_out", ctypes.c_void_p),
                ("scores_out", ctypes.c_void_p), ("dev_status", ctypes.c_void_p)]


class seer_append_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("q_out", ctypes.c_void_p),
                ("cu_tokens", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("rope", ctypes.c_void_p), ("total_tokens", ctypes.c_int32),
                ("max_new", ctypes.c_int32), ("max_position", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("cache_type", ctypes.c_int32), ("k_pool", ctypes.c_void_p),
                ("v_pool", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("seqlens", ctypes.c_void_p), ("kbar", ctypes.c_void_p),
                ("dev_status", ctypes.c_void_p)]


class seer_cache_attn_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("cache_type", ctypes.c_int32),
                ("num_splits", ctypes.c_int32), ("k_pool", ctypes.c_void_p),
                ("v_pool", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("seqlens", ctypes.c_void_p), ("idx", ctypes.c_void_p),
                ("n_sel", ctypes.c_void_p), ("k_max", ctypes.c_int32),
                ("window", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("out", ctypes.c_void_p),
                ("lse_out", ctypes.c_void_p), ("dev_status", ctypes.c_void_p)]


class seer_window_prefill_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("cu_tokens", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("seqlens", ctypes.c_void_p), ("total_tokens", ctypes.c_int32),
                ("max_new", ctypes.c_int32), ("window", ctypes.c_int32),
                ("sinks", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("out", ctypes.c_void_p), ("lse_out", ctypes.c_void_p),
                ("dev_status", ctypes.c_void_p)]


_P = ctypes.c_void_p
_D = ctypes.POINTER(seer_dims)
_I = ctypes.c_int32
_SIGS = {
    "seer_version": (_I, []),
    "seer_status_string": (ctypes.c_char_p, [_I]),
    "seer_last_cuda_error": (ctypes.c_char_p, []),
    "seer_dims_default": (_I, [_I, _I, _I, _I, _I, _I, ctypes.c_int64, _D]),
    "seer_k_from_sparsity": (_I, [_I, _I, ctypes.POINTER(_I)]),
    "seer_k_from_budget": (_I, [_I, _I, _I, ctypes.POINTER(_I)]),
    "seer_fill_k": (_I, [_D, _P, _I, _I, _P, _P]),
    "seer_default_splits": (_I, [_D, _I, _I]),
    "seer_step_workspace_bytes": (ctypes.c_size_t, [_D, _I, _I]),
    "seer_pool_keys": (_I, [_D, _P, _P, _P, _I, _P, _P, _P]),
    "seer_gate_scores": (_I, [_D, _P, _P, _P, _P, ctypes.c_float, _P, _P, _P]),
    "seer_block_select": (_I, [_D, _P, _P, _P, _I, _I, _P, _P, _P, _P]),
    "seer_block_select_unified": (_I, [_D, _P, _P, _P, _I, _I, _P, _P, _P, _P]),
    "seer_sparse_decode": (_I, [_D, _P, _P, _P, _P, _P, _P, _P, _I, _I, ctypes.c_float, _P, _P,
                                _P, _P, _P]),
    "seer_combine": (_I, [_D, _P, _P, _I, _P, _P, _P]),
    "seer_decode_step": (_I, [_D, ctypes.POINTER(seer_step_args), _P]),
    "seer_decode_step_host": (_I, [_D, ctypes.POINTER(seer_step_args), _P, _P, _P, _P]),
    "seer_host_ptr_mapped": (_I, [_P]),
    "seer_decode_step_noalloc": (_I, [_D, ctypes.POINTER(seer_step_args), _P]),
    "seer_decode_step_fused": (_I, [_D, ctypes.POINTER(seer_step_args), _P]),
    "seer_step_workspace_init": (_I, [_D, _I, _I, _P, ctypes.c_size_t, _P]),
    "seer_prefill_k_max": (_I, [_D, _I, _I]),
    "seer_prefill_workspace_bytes": (ctypes.c_size_t, [_D, _I]),
    "seer_prefill": (_I, [_D, ctypes.POINTER(seer_prefill_args), _P]),
    "seer_prefill_attention": (_I, [_D, ctypes.POINTER(seer_prefill_args), _P, _P, _P]),
    "seer_block_lse_elems": (ctypes.c_size_t, [_D]),
    "seer_sparse_decode_mass": (_I, [_D, _P, _P, _P, _P, _P, _P, _P, _I, _I, ctypes.c_float, _P, _P,
                                     _P, _P, _P, _P]),
    "seer_block_mass": (_I, [_D, _P, _P, _I, _P, _P, _P, _P, _P]),
    "seer_rope_table": (_I, [_I, _I, ctypes.c_double, _P, _P]),
    "seer_append_rope": (_I, [_D, ctypes.POINTER(seer_append_args), _P]),
    "seer_sparse_decode_q8_splits": (_I, [_D, _I]),
    "seer_window_decode_splits": (_I, [_D, _I, _I]),
    "seer_split_workspace_bytes": (ctypes.c_size_t, [_D, _I]),
    "seer_sparse_decode_q8": (_I, [_D, ctypes.POINTER(seer_cache_attn_args), _P]),
    "seer_window_decode": (_I, [_D, ctypes.POINTER(seer_cache_attn_args), _P]),
    "seer_window_prefill": (_I, [_D, ctypes.POINTER(seer_window_prefill_args), _P]),
}

_lib_handle = None


def _lib():
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m block_sparse_attention_step_b200.build` (no fallback exists)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib_handle = lib
    return _lib_handle


def library():
    """The loaded ctypes library (loads it on first call)."""
    return _lib()


def _check(fn: str, status: int):
    if status != SEER_OK:
        raise SeerError(fn, status)


def _ptr(t, dtype=None, name="tensor", allow_none=False, device=True):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_dims(batch, num_q_heads, num_kv_heads, head_dim, block_size, max_blocks, num_pages,
              stride_page=None, stride_token=None, stride_head=None) -> seer_dims:
    d = seer_dims()
    _check("seer_dims_default", _lib().seer_dims_default(batch, num_q_heads, num_kv_heads, head_dim,
                                                         block_size, max_blocks, num_pages,
                                                         ctypes.byref(d)))
    if stride_page is not None:
        d.stride_page, d.stride_token, d.stride_head = stride_page, stride_token, stride_head
    return d


def version() -> int:
    return _lib().seer_version()


def seer_k_from_sparsity(nb: int, sparsity_permille: int) -> int:
    k = ctypes.c_int32()
    _check("seer_k_from_sparsity", _lib().seer_k_from_sparsity(nb, sparsity_permille, ctypes.byref(k)))
    return k.value


def seer_k_from_budget(nb: int, budget_tokens: int, block_size: int) -> int:
    k = ctypes.c_int32()
    _check("seer_k_from_budget", _lib().seer_k_from_budget(nb, budget_tokens, block_size, ctypes.byref(k)))
    return k.value


def seer_fill_k(d, seqlens, sparsity_permille, budget_tokens, k_per_seq, stream=None):
    _check("seer_fill_k", _lib().seer_fill_k(ctypes.byref(d), _ptr(seqlens, torch.int32, "seqlens"),
                                             sparsity_permille, budget_tokens,
                                             _ptr(k_per_seq, torch.int32, "k_per_seq"), _stream(stream)))


def seer_default_splits(d, k_max: int, num_sms: int = 0) -> int:
    return _lib().seer_default_splits(ctypes.byref(d), k_max, num_sms)


def seer_step_workspace_bytes(d, k_max: int, num_splits: int) -> int:
    return _lib().seer_step_workspace_bytes(ctypes.byref(d), k_max, num_splits)


def seer_pool_keys(d, k_pool, page_table, seqlens, incremental, kbar, dev_status=None, stream=None):
    _check("seer_pool_keys", _lib().seer_pool_keys(
        ctypes.byref(d), _ptr(k_pool, torch.bfloat16, "k_pool"),
        _ptr(page_table, torch.int32, "page_table", allow_none=True),
        _ptr(seqlens, torch.int32, "seqlens"), int(incremental), _ptr(kbar, torch.float32, "kbar"),
        _ptr(dev_status, torch.int32, "dev_status", allow_none=True), _stream(stream)))


def seer_gate_scores(d, q, w_gate, kbar, seqlens, gate_scale, scores, dev_status=None, stream=None):
    _check("seer_gate_scores", _lib().seer_gate_scores(
        ctypes.byref(d), _ptr(q, torch.bfloat16, "q"), _ptr(w_gate, torch.float32, "w_gate"),
        _ptr(kbar, torch.float32, "kbar"), _ptr(seqlens, torch.int32, "seqlens"), float(gate_scale),
        _ptr(scores, torch.float32, "scores"),
        _ptr(dev_status, torch.int32, "dev_status", allow_none=True), _stream(stream)))


def seer_block_select(d, scores, seqlens, k_per_seq, force_newest, k_max, idx, n_sel,
                      dev_status=None, stream=None):
    _check("seer_block_select", _lib().seer_block_select(
        ctypes.byref(d), _ptr(scores, torch.float32, "scores"), _ptr(seqlens, torch.int32, "seqlens"),
        _ptr(k_per_seq, torch.int32, "k_per_seq"), int(bool(force_newest)), int(k_max),
        _ptr(idx, torch.int32, "idx"), _ptr(n_sel, torch.int32, "n_sel"),
        _ptr(dev_status, torch.int32, "dev_status", allow_none=True), _stream(stream)))


def seer_block_select_unified(d, scores, seqlens, k_per_seq, force_newest, k_max, idx, n_sel,
                      dev_status=None, stream=None):
    _check("seer_block_select_unified", _lib().seer_block_select_unified(
        ctypes.byref(d), _ptr(scores, torch.float32, "scores"), _ptr(seqlens, torch.int32, "seqlens"),
        _ptr(k_per_seq, torch.int32, "k_per_seq"), int(bool(force_newest)), int(k_max),
        _ptr(idx, torch.int32, "idx"), _ptr(n_sel, torch.int32, "n_sel"),
        _ptr(dev_status, torch.int32, "dev_status", allow_none=True), _stream(stream)))


def seer_sparse_decode(d, q, k_pool, v_pool, page_table, seqlens, idx, n_sel, k_max, num_splits,
                       softmax_scale, o_part, lse_part, dev_status=None, stream=None, *,
                       work_counter=None):
    """work_counter: None (round-robin items) or 2 zeroed int32 words on the device."""
    _check("seer_sparse_decode", _lib().seer_sparse_decode(
        ctypes.byref(d), _ptr(q, torch.bfloat16, "q"), _ptr(k_pool, torch.bfloat16, "k_pool"),
        _ptr(v_pool, torch.bfloat16, "v_pool"),
        _ptr(page_table, torch.int32, "page_table", allow_none=True),
        _ptr(seqlens, torch.int32, "seqlens"), _ptr(idx, torch.int32, "idx"),
        _ptr(n_sel, torch.int32, "n_sel"), int(k_max), int(num_splits), float(softmax_scale),
        _ptr(o_part, torch.float32, "o_part"), _ptr(lse_part, torch.float32, "lse_part"),
        _ptr(work_counter, torch.int32, "work_counter", allow_none=True),
        _ptr(dev_status, torch.int32, "dev_status", allow_none=True), _stream(stream)))


def seer_combine(d, o_part, lse_part, num_splits, out, lse_out=None, stream=None):
    _check("seer_combine", _lib().seer_combine(
        ctypes.byref(d), _ptr(o_part, torch.float32, "o_part"),
        _ptr(lse_part, torch.float32, "lse_part"), int(num_splits),
        _ptr(out, torch.bfloat16, "out"), _ptr(lse_out, torch.float32, "lse_out", allow_none=True),
        _stream(stream)))


def step_args(q, k_pool, v_pool, page_table, seqlens, w_gate, kbar, k_per_seq, *, update_kbar,
              force_newest, k_max, num_splits, gate_scale, softmax_scale, workspace, out,
              lse_out=None, dev_status=None, block_lse=None, block_mass=None,
              unified_heads=False, k_new=None, v_new=None) -> seer_step_args:
    a = seer_step_args()
    a.q = _ptr(q, torch.bfloat16, "q", allow_none=True)
    a.k_pool = _ptr(k_pool, torch.bfloat16, "k_pool")
    a.v_pool = _ptr(v_pool, torch.bfloat16, "v_pool")
    a.page_table = _ptr(page_table, torch.int32, "page_table", allow_none=True)
    a.seqlens = _ptr(seqlens, torch.int32, "seqlens")
    a.w_gate = _ptr(w_gate, torch.float32, "w_gate")
    a.kbar = _ptr(kbar, torch.float32, "kbar")
    a.k_per_seq = _ptr(k_per_seq, torch.int32, "k_per_seq")
    a.update_kbar = int(update_kbar)
    a.force_newest = int(bool(force_newest))
    a.k_max = int(k_max)
    a.num_splits = int(num_splits)
    a.gate_scale = float(gate_scale)
    a.softmax_scale = float(softmax_scale)
    a.workspace = _ptr(workspace, torch.uint8, "workspace")
    a.workspace_bytes = workspace.numel()
    a.out = _ptr(out, torch.bfloat16, "out")
    a.lse_out = _ptr(lse_out, torch.float32, "lse_out", allow_none=True)
    a.dev_status = _ptr(dev_status, torch.int32, "dev_status", allow_none=True)
    a.block_lse = _ptr(block_lse, torch.float32, "block_lse", allow_none=True)
    a.block_mass = _ptr(block_mass, torch.float32, "block_mass", allow_none=True)
    a.unified_heads = int(bool(unified_heads))
    a.k_new = _ptr(k_new, torch.bfloat16, "k_new", allow_none=True)
    a.v_new = _ptr(v_new, torch.bfloat16, "v_new", allow_none=True)
    return a


def seer_decode_step(d, args: seer_step_args, stream=None):
    _check("seer_decode_step", _lib().seer_decode_step(ctypes.byref(d), ctypes.byref(args),
                                                       _stream(stream)))


def seer_decode_step_fused(d, args: seer_step_args, stream=None):
    _check("seer_decode_step_fused", _lib().seer_decode_step_fused(ctypes.byref(d),
                                                                   ctypes.byref(args),
                                                                   _stream(stream)))


def seer_step_workspace_init(d, k_max, num_splits, workspace, stream=None):
    _check("seer_step_workspace_init", _lib().seer_step_workspace_init(
        ctypes.byref(d), int(k_max), int(num_splits), _ptr(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream)))


def seer_decode_step_host(d, args: seer_step_args, q_host, q_dev, out_host, stream=None):
    _check("seer_decode_step_host", _lib().seer_decode_step_host(
        ctypes.byref(d), ctypes.byref(args), _ptr(q_host, torch.bfloat16, "q_host", device=False),
        _ptr(q_dev, torch.bfloat16, "q_dev"), _ptr(out_host, torch.bfloat16, "out_host", device=False),
        _stream(stream)))


def seer_host_ptr_mapped(t) -> bool:
    """True if seer_decode_step_host accesses this host tensor directly from
    its kernels (pinned and mapped into the device), False if it copies."""
    if t.is_cuda:
        raise ValueError("expected a host tensor")
    return bool(_lib().seer_host_ptr_mapped(ctypes.c_void_p(t.data_ptr())))


def seer_decode_step_noalloc(d, args: seer_step_args, stream=None):
    """The step with the library's own fixed 16 MiB device scratch instead of
    ``args.workspace`` (for callers that cannot allocate device memory)."""
    _check("seer_decode_step_noalloc", _lib().seer_decode_step_noalloc(
        ctypes.byref(d), ctypes.byref(args), _stream(stream)))


def seer_block_lse_elems(d) -> int:
    return _lib().seer_block_lse_elems(ctypes.byref(d))


def seer_sparse_decode_mass(d, q, k_pool, v_pool, page_table, seqlens, idx, n_sel, k_max,
                            num_splits, softmax_scale, o_part, lse_part, block_lse,
                            dev_status=None, stream=None, *, work_counter=None):
    _check("seer_sparse_decode_mass", _lib().seer_sparse_decode_mass(
        ctypes.byref(d), _ptr(q, torch.bfloat16, "q"), _ptr(k_pool, torch.bfloat16, "k_pool"),
        _ptr(v_pool, torch.bfloat16, "v_pool"),
        _ptr(page_table, torch.int32, "page_table", allow_none=True),
        _ptr(seqlens, torch.int32, "seqlens"), _ptr(idx, torch.int32, "idx"),
        _ptr(n_sel, torch.int32, "n_sel"), int(k_max), int(num_splits), float(softmax_scale),
        _ptr(o_part, torch.float32, "o_part"), _ptr(lse_part, torch.float32, "lse_part"),
        _ptr(block_lse, torch.float32, "block_lse"),
        _ptr(work_counter, torch.int32, "work_counter", allow_none=True),
        _ptr(dev_status, torch.int32, "dev_status", allow_none=True), _stream(stream)))


def seer_block_mass(d, idx, n_sel, k_max, seqlens, block_lse, lse, mass, stream=None):
    _check("seer_block_mass", _lib().seer_block_mass(
        ctypes.byref(d), _ptr(idx, torch.int32, "idx"), _ptr(n_sel, torch.int32, "n_sel"),
        int(k_max), _ptr(seqlens, torch.int32, "seqlens"),
        _ptr(block_lse, torch.float32, "block_lse"), _ptr(lse, torch.float32, "lse"),
        _ptr(mass, torch.float32, "mass"), _stream(stream)))


def seer_prefill_k_max(d, sparsity_permille, budget_tokens):
    return _lib().seer_prefill_k_max(ctypes.byref(d), int(sparsity_permille), int(budget_tokens))


def seer_prefill_workspace_bytes(d, k_max):
    return _lib().seer_prefill_workspace_bytes(ctypes.byref(d), int(k_max))


def seer_prefill_attention(d, q, k_pool, v_pool, page_table, seqlens, idx, n_sel, *, k_max,
                           softmax_scale, out, lse_out=None, dev_status=None, stream=None):
    a = seer_prefill_args()
    a.q = _ptr(q, torch.bfloat16, "q")
    a.k_pool = _ptr(k_pool, torch.bfloat16, "k_pool")
    a.v_pool = _ptr(v_pool, torch.bfloat16, "v_pool")
    a.page_table = _ptr(page_table, torch.int32, "page_table", allow_none=True)
    a.seqlens = _ptr(seqlens, torch.int32, "seqlens")
    a.k_max = int(k_max)
    a.softmax_scale = float(softmax_scale)
    a.out = _ptr(out, torch.bfloat16, "out")
    a.lse_out = _ptr(lse_out, torch.float32, "lse_out", allow_none=True)
    a.dev_status = _ptr(dev_status, torch.int32, "dev_status", allow_none=True)
    _check("seer_prefill_attention", _lib().seer_prefill_attention(
        ctypes.byref(d), ctypes.byref(a), _ptr(idx, torch.int32, "idx"),
        _ptr(n_sel, torch.int32, "n_sel"), _stream(stream)))


def seer_prefill(d, q, k_pool, v_pool, page_table, seqlens, w_gate, kbar, *, pool_keys,
                 sparsity_permille, budget_tokens, k_max, gate_scale, softmax_scale, workspace,
                 out, lse_out=None, scores_out=None, dev_status=None, stream=None):
    a = seer_prefill_args()
    a.q = _ptr(q, torch.bfloat16, "q")
    a.k_pool = _ptr(k_pool, torch.bfloat16, "k_pool")
    a.v_pool = _ptr(v_pool, torch.bfloat16, "v_pool")
    a.page_table = _ptr(page_table, torch.int32, "page_table", allow_none=True)
    a.seqlens = _ptr(seqlens, torch.int32, "seqlens")
    a.w_gate = _ptr(w_gate, torch.float32, "w_gate")
    a.kbar = _ptr(kbar, torch.float32, "kbar")
    a.pool_keys = int(bool(pool_keys))
    a.sparsity_permille = int(sparsity_permille)
    a.budget_tokens = int(budget_tokens)
    a.k_max = int(k_max)
    a.gate_scale = float(gate_scale)
    a.softmax_scale = float(softmax_scale)
    a.workspace = _ptr(workspace, torch.uint8, "workspace")
    a.workspace_bytes = workspace.numel()
    a.out = _ptr(out, torch.bfloat16, "out")
    a.lse_out = _ptr(lse_out, torch.float32, "lse_out", allow_none=True)
    a.scores_out = _ptr(scores_out, torch.float32, "scores_out", allow_none=True)
    a.dev_status = _ptr(dev_status, torch.int32, "dev_status", allow_none=True)
    _check("seer_prefill", _lib().seer_prefill(ctypes.byref(d), ctypes.byref(a), _stream(stream)))



# ------------------------------------------------------------ paged KV cache
def _keep(a, **tensors):
    """Argument blocks of the cache operators hold on to their tensors, by name,
    and remember the device these are on."""
    live = {name: t for name, t in tensors.items() if t is not None}
    devices = {t.device for t in live.values()}
    if len(devices) > 1:
        raise ValueError(f"tensors on more than one device: {sorted(map(str, devices))}")
    a.tensors = live
    a.device = devices.pop().index
    a.fits = None  # the dims and arguments that the tensors were last found to fit
    return a


def _shapes(d, a):
    """Shape that an operator takes each tensor of its argument block for (the
    pools, which have strides of their own: elements)."""
    B, Hq, Hkv, D, blocks = d.batch, d.num_q_heads, d.num_kv_heads, d.head_dim, d.max_blocks
    pool = ((d.num_pages - 1) * d.stride_page + (d.block_size - 1) * d.stride_token
            + (Hkv - 1) * d.stride_head + D)
    shapes = dict(k_pool=(pool,), v_pool=(pool,), k_scale=(d.num_pages, Hkv),
                  v_scale=(d.num_pages, Hkv), page_table=(B, blocks), seqlens=(B,),
                  cu_tokens=(B + 1,), dev_status=(1,))
    if isinstance(a, seer_cache_attn_args):
        rows = B
        shapes.update(idx=(B, Hkv, a.k_max), n_sel=(B, Hkv), lse_out=(B, Hq),
                      workspace=(0,))  # the library checks its bytes
    else:
        rows = a.total_tokens
        shapes.update(positions=(rows,), kbar=(B, Hkv, blocks, D), lse_out=(Hq, rows),
                      rope=(getattr(a, "max_position", 0), getattr(a, "rotary_dim", 0)))
    shapes.update(q=(rows, Hq, D), q_out=(rows, Hq, D), out=(rows, Hq, D), k_new=(rows, Hkv, D),
                  v_new=(rows, Hkv, D))
    return shapes


def _check_sizes(fn: str, d, a):
    """No tensor is smaller than the dims and the other arguments say (the
    kernels take their word for it), and none has other inner extents.  One of
    another number of dimensions counts by its elements."""
    shapes = _shapes(d, a)
    for name, t in a.tensors.items():
        want, got = shapes[name], tuple(t.shape)
        if t.numel() < math.prod(want):
            raise ValueError(f"{fn}: {name} has {t.numel()} elements, the dims ask for "
                             f"{math.prod(want)}")
        rows = isinstance(a, seer_append_args) and name in ("q", "q_out", "k_new", "v_new")
        for i in range(1, len(want) if len(got) == len(want) else 0):
            # behind a single row another extent moves nothing (strided rows apart)
            if got[i] != want[i] and (rows or math.prod(want[:i]) > 1):
                raise ValueError(f"{fn}: {name} is {list(got)}, the dims ask for {list(want)}")


def _call(fn: str, d, a, stream):
    """A cache operator on its tensors' device, which has to be the current one."""
    device = torch.cuda.current_device()
    if a.device != device:
        raise ValueError(f"{fn}: tensors on cuda:{a.device}, current device is cuda:{device}")
    asked = (bytes(d), bytes(a))
    if a.fits != asked:  # once for each content of the two: a call per step repeats them
        _check_sizes(fn, d, a)
        a.fits = asked
    raw = torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)
    status = getattr(_lib_handle or _lib(), fn)(ctypes.byref(d), ctypes.byref(a), raw)
    if status != SEER_OK:
        raise SeerError(fn, status)


def _cache(a, k_pool, v_pool, k_scale, v_scale):
    if k_pool.dtype not in _CACHE_TYPES:
        raise TypeError(f"k_pool must be bfloat16, float8_e4m3fn or int8, got {k_pool.dtype}")
    a.cache_type = _CACHE_TYPES[k_pool.dtype]
    a.k_pool = _ptr(k_pool, k_pool.dtype, "k_pool")
    a.v_pool = _ptr(v_pool, k_pool.dtype, "v_pool")
    eight = a.cache_type != CACHE_BF16
    if not eight and (k_scale is not None or v_scale is not None):
        raise ValueError("a bfloat16 cache has no scales")
    a.k_scale = _ptr(k_scale, torch.float32, "k_scale", allow_none=not eight)
    a.v_scale = _ptr(v_scale, torch.float32, "v_scale", allow_none=not eight)


def _rows(t, name):
    """(pointer, elements between tokens) of [T][H][D] bf16 rows whose heads
    are D apart; the tokens may be further apart (a fused projection)."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens][heads][head_dim]")
    T, H, D = t.shape
    if t.numel() and (t.stride(2) != 1 or (H > 1 and t.stride(1) != D)
                      or (T > 1 and t.stride(0) < H * D)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return ctypes.c_void_p(t.data_ptr()), (t.stride(0) if T > 1 else H * D)


def seer_rope_table(max_position: int, rotary_dim: int, base: float = 10000.0, table=None,
                    device=None, stream=None):
    """[max_position][rotary_dim] fp32 table of a position rotation (cosines,
    then sines), allocated unless given."""
    if table is None:
        table = torch.empty((max_position, rotary_dim), dtype=torch.float32,
                            device=device or torch.device("cuda", torch.cuda.current_device()))
    if tuple(table.shape) != (max_position, rotary_dim):
        raise ValueError("table must be [max_position][rotary_dim]")
    at = _ptr(table, torch.float32, "table")
    if table.device.index != torch.cuda.current_device():
        raise ValueError(f"seer_rope_table: table on {table.device}, current device is "
                         f"cuda:{torch.cuda.current_device()}")
    _check("seer_rope_table", _lib().seer_rope_table(
        int(max_position), int(rotary_dim), float(base), at, _stream(stream)))
    return table


def append_args(k_new, v_new, k_pool, v_pool, page_table, seqlens, *, q=None, q_out=None,
                rope=None, interleaved=False, cu_tokens=None, max_new=1, positions=None,
                k_scale=None, v_scale=None, kbar=None, dev_status=None) -> seer_append_args:
    """Arguments of seer_append_rope: [T][heads][D] bf16 rows of q (optional),
    k and v, a cache in bfloat16, float8_e4m3fn or int8 (with its scales), and
    the rotation table (None: no rotation)."""
    a = seer_append_args()
    a.k_new, a.k_stride = _rows(k_new, "k_new")
    a.v_new, a.v_stride = _rows(v_new, "v_new")
    if k_new.shape != v_new.shape:
        raise ValueError("k_new and v_new differ in shape")
    if q is not None:
        a.q, a.q_stride = _rows(q, "q")
        if q.shape[0] != k_new.shape[0]:
            raise ValueError("q and k_new differ in tokens")
        if q_out is None:
            raise ValueError("q_out is required with q")
        if q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
        if q_out.data_ptr() == q.data_ptr():
            a.q_out, out_stride = _rows(q_out, "q_out")
            if out_stride != a.q_stride:
                raise ValueError("q_out over q must have q's strides")
        else:
            a.q_out = _ptr(q_out, torch.bfloat16, "q_out")
    _cache(a, k_pool, v_pool, k_scale, v_scale)
    a.cu_tokens = _ptr(cu_tokens, torch.int32, "cu_tokens", allow_none=True)
    a.positions = _ptr(positions, torch.int32, "positions", allow_none=True)
    a.rope = _ptr(rope, torch.float32, "rope", allow_none=True)
    a.total_tokens = k_new.shape[0]
    a.max_new = int(max_new)
    if rope is not None:
        a.max_position, a.rotary_dim = rope.shape
    a.interleaved = int(bool(interleaved))
    a.page_table = _ptr(page_table, torch.int32, "page_table", allow_none=True)
    a.seqlens = _ptr(seqlens, torch.int32, "seqlens")
    a.kbar = _ptr(kbar, torch.float32, "kbar", allow_none=True)
    a.dev_status = _ptr(dev_status, torch.int32, "dev_status", allow_none=True)
    return _keep(a, k_new=k_new, v_new=v_new, k_pool=k_pool, v_pool=v_pool, page_table=page_table,
                 seqlens=seqlens, q=q, q_out=q_out, rope=rope, cu_tokens=cu_tokens,
                 positions=positions, k_scale=k_scale, v_scale=v_scale, kbar=kbar,
                 dev_status=dev_status)


def seer_append_rope(d, args: seer_append_args, stream=None):
    """Rotate new q / k rows and append k / v to the paged cache."""
    _call("seer_append_rope", d, args, stream)


def seer_sparse_decode_q8_splits(d, k_max: int) -> int:
    return _lib().seer_sparse_decode_q8_splits(ctypes.byref(d), int(k_max))


def seer_window_decode_splits(d, window: int, sinks: int) -> int:
    return _lib().seer_window_decode_splits(ctypes.byref(d), int(window), int(sinks))


def seer_split_workspace_bytes(d, num_splits: int) -> int:
    return _lib().seer_split_workspace_bytes(ctypes.byref(d), int(num_splits))


def _cache_attn(q, k_pool, v_pool, page_table, seqlens, k_scale, v_scale, num_splits, workspace,
                softmax_scale, out, lse_out, dev_status, **more):
    a = seer_cache_attn_args()
    a.q = _ptr(q, torch.bfloat16, "q")
    _cache(a, k_pool, v_pool, k_scale, v_scale)
    a.num_splits = int(num_splits)
    a.page_table = _ptr(page_table, torch.int32, "page_table", allow_none=True)
    a.seqlens = _ptr(seqlens, torch.int32, "seqlens")
    a.softmax_scale = float(softmax_scale)
    if workspace is not None:
        a.workspace = _ptr(workspace, torch.uint8, "workspace")
        a.workspace_bytes = workspace.numel()
    a.out = _ptr(out, torch.bfloat16, "out")
    a.lse_out = _ptr(lse_out, torch.float32, "lse_out", allow_none=True)
    a.dev_status = _ptr(dev_status, torch.int32, "dev_status", allow_none=True)
    return _keep(a, q=q, k_pool=k_pool, v_pool=v_pool, page_table=page_table, seqlens=seqlens,
                 k_scale=k_scale, v_scale=v_scale, workspace=workspace, out=out, lse_out=lse_out,
                 dev_status=dev_status, **more)


def sparse_decode_q8_args(q, k_pool, v_pool, page_table, seqlens, idx, n_sel, *, k_scale, v_scale,
                          k_max, num_splits, softmax_scale, out, workspace=None, lse_out=None,
                          dev_status=None) -> seer_cache_attn_args:
    """Arguments of seer_sparse_decode_q8 (float8_e4m3fn or int8 pools)."""
    a = _cache_attn(q, k_pool, v_pool, page_table, seqlens, k_scale, v_scale, num_splits,
                    workspace, softmax_scale, out, lse_out, dev_status, idx=idx, n_sel=n_sel)
    a.idx = _ptr(idx, torch.int32, "idx")
    a.n_sel = _ptr(n_sel, torch.int32, "n_sel")
    a.k_max = int(k_max)
    return a


def window_decode_args(q, k_pool, v_pool, page_table, seqlens, *, window, sinks, num_splits,
                       softmax_scale, out, k_scale=None, v_scale=None, workspace=None,
                       lse_out=None, dev_status=None) -> seer_cache_attn_args:
    """Arguments of seer_window_decode (bfloat16, float8_e4m3fn or int8 pools)."""
    a = _cache_attn(q, k_pool, v_pool, page_table, seqlens, k_scale, v_scale, num_splits,
                    workspace, softmax_scale, out, lse_out, dev_status)
    a.window = int(window)
    a.sinks = int(sinks)
    return a


def seer_sparse_decode_q8(d, args: seer_cache_attn_args, stream=None):
    """Block-sparse decode attention over an 8-bit cache, out and lse in one call."""
    _call("seer_sparse_decode_q8", d, args, stream)


def seer_window_decode(d, args: seer_cache_attn_args, stream=None):
    """Sliding-window decode attention with sink tokens, out and lse in one call."""
    _call("seer_window_decode", d, args, stream)


def window_prefill_args(q, k_pool, v_pool, page_table, seqlens, *, window, sinks, softmax_scale,
                        out, cu_tokens=None, max_new=1, lse_out=None,
                        dev_status=None) -> seer_window_prefill_args:
    """Arguments of seer_window_prefill: q and out [T][Hq][D] bf16, lse_out
    [Hq][T] fp32, bfloat16 pools."""
    a = seer_window_prefill_args()
    a.q = _ptr(q, torch.bfloat16, "q")
    a.k_pool = _ptr(k_pool, torch.bfloat16, "k_pool")
    a.v_pool = _ptr(v_pool, torch.bfloat16, "v_pool")
    a.cu_tokens = _ptr(cu_tokens, torch.int32, "cu_tokens", allow_none=True)
    a.page_table = _ptr(page_table, torch.int32, "page_table", allow_none=True)
    a.seqlens = _ptr(seqlens, torch.int32, "seqlens")
    a.total_tokens = q.shape[0]
    a.max_new = int(max_new)
    a.window = int(window)
    a.sinks = int(sinks)
    a.softmax_scale = float(softmax_scale)
    a.out = _ptr(out, torch.bfloat16, "out")
    a.lse_out = _ptr(lse_out, torch.float32, "lse_out", allow_none=True)
    a.dev_status = _ptr(dev_status, torch.int32, "dev_status", allow_none=True)
    return _keep(a, q=q, k_pool=k_pool, v_pool=v_pool, cu_tokens=cu_tokens, page_table=page_table,
                 seqlens=seqlens, out=out, lse_out=lse_out, dev_status=dev_status)


def seer_window_prefill(d, args: seer_window_prefill_args, stream=None):
    """Sliding-window attention with sink tokens for a ragged chunk of query tokens."""
    _call("seer_window_prefill", d, args, stream)
