"""Paged decode attention for GB300: Python binding of libzl_decode_attn.so.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of the library (declared in include/zl_decode_attn.h). There is no CPU
or PyTorch fallback; if the library is missing or fails to load, every call
raises.

    import paged_decode_attention_gqa_gb300 as zl
    out = zl.decode_attn(q, k_pool, v_pool, block_table, seq_lens,
                         page_size=16, scale=128 ** -0.5)

Tensors are torch CUDA tensors (PyTorch provides device memory and streams).
"""

from __future__ import annotations

import contextlib
import ctypes
import math
import os
import re
import struct
import threading

import torch

from ._build import LIB_PATH, build  # noqa: F401  (build() is the public build step)

__all__ = [
    "ZlError", "Params", "AppendParams", "ScoreParams", "EvictParams", "CommitParams",
    "AppendQ4Params", "ReadQ4Params", "DecodeQ4Params", "NormRopeParams", "lib",
    "decode_attn", "decode_attn_mla", "kv_append", "kv_evict", "kv_commit", "tree_mask",
    "decode_attn_q4", "kv_append_q4", "kv_read_q4", "qk_norm_rope", "Rope", "rope_frequencies",
    "Q4_ROW_BYTES",
    "workspace_size", "workspace_size_mla", "workspace_size_ex", "call", "call_ex",
    "call_noalloc", "build", "LIB_PATH",
    "DEVERR_BAD_PAGE", "DEVERR_BAD_SEQ_LEN", "DEVERR_TIMEOUT", "DEVERR_BAD_PATH", "HEADER",
    "declared_symbols",
]

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "zl_decode_attn.h")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA = range(5)
SINGLE_LAUNCH = 1  # ZL_DECODE_SINGLE_LAUNCH
TEST_STALL = 0x80000000  # ZL_DECODE_TEST_STALL (failure-detection test hook)
DEVERR_BAD_PAGE, DEVERR_BAD_SEQ_LEN, DEVERR_TIMEOUT, DEVERR_BAD_PREFIX = 1, 2, 4, 8
DEVERR_BAD_PATH = 16
NOALLOC_WORKSPACE_BYTES = 8 << 20  # ZL_NOALLOC_WORKSPACE_BYTES
Q4_ROW_BYTES = 144  # ZL_Q4_ROW_BYTES
CACHE_NONE, CACHE_BF16, CACHE_Q4 = range(3)  # zl_cache_kind


class ZlError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{msg} (zl_status {status})")
        self.status = status


class Params(ctypes.Structure):
    """Mirror of zl_decode_attn_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("q", ctypes.c_void_p),
        ("k_pool", ctypes.c_void_p),
        ("v_pool", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("block_table", ctypes.c_void_p),
        ("block_table_stride", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p),
        ("B", ctypes.c_int32),
        ("q_len", ctypes.c_int32),
        ("Hq", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("D_qk", ctypes.c_int32),
        ("D_v", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("err_flags", ctypes.c_void_p),
        ("num_ctas", ctypes.c_int32),
        ("attn_begin", ctypes.c_void_p),
        ("attn_end", ctypes.c_void_p),
        ("flags", ctypes.c_uint32),
        ("shared_prefix_pages", ctypes.c_int32),
        ("k_new", ctypes.c_void_p),
        ("v_new", ctypes.c_void_p),
    ]


class AppendParams(ctypes.Structure):
    """Mirror of zl_kv_append_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("k_new", ctypes.c_void_p),
        ("v_new", ctypes.c_void_p),
        ("k_pool", ctypes.c_void_p),
        ("v_pool", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("block_table", ctypes.c_void_p),
        ("block_table_stride", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p),
        ("B", ctypes.c_int32),
        ("q_len", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("D_k", ctypes.c_int32),
        ("D_v", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("err_flags", ctypes.c_void_p),
    ]


class ScoreParams(ctypes.Structure):
    """Mirror of zl_score_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("softcap", ctypes.c_float),
        ("window", ctypes.c_int32),
        ("alibi_slopes", ctypes.c_void_p),
        ("tree_mask", ctypes.c_void_p),
        ("weights", ctypes.c_void_p),
        ("weights_seq_stride", ctypes.c_int64),
        ("weights_head_stride", ctypes.c_int64),
        ("weights_tokens", ctypes.c_int32),
        ("weights_decay", ctypes.c_float),
    ]


class EvictParams(ctypes.Structure):
    """Mirror of zl_kv_evict_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("k_pool", ctypes.c_void_p),
        ("v_pool", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("block_table", ctypes.c_void_p),
        ("block_table_stride", ctypes.c_int64),
        ("dst_block_table", ctypes.c_void_p),
        ("dst_block_table_stride", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p),
        ("new_lens", ctypes.c_void_p),
        ("kept", ctypes.c_void_p),
        ("weights", ctypes.c_void_p),
        ("weights_seq_stride", ctypes.c_int64),
        ("weights_head_stride", ctypes.c_int64),
        ("weights_out", ctypes.c_void_p),
        ("weights_out_seq_stride", ctypes.c_int64),
        ("weights_out_head_stride", ctypes.c_int64),
        ("weights_tokens", ctypes.c_int32),
        ("B", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("D_k", ctypes.c_int32),
        ("D_v", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("budget", ctypes.c_int32),
        ("sink", ctypes.c_int32),
        ("recent", ctypes.c_int32),
        ("err_flags", ctypes.c_void_p),
        ("weights_clear", ctypes.c_int32),
    ]


class CommitParams(ctypes.Structure):
    """Mirror of zl_kv_commit_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("k_pool", ctypes.c_void_p),
        ("v_pool", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("block_table", ctypes.c_void_p),
        ("block_table_stride", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p),
        ("path", ctypes.c_void_p),
        ("path_stride", ctypes.c_int64),
        ("accepted", ctypes.c_void_p),
        ("new_lens", ctypes.c_void_p),
        ("path_len", ctypes.c_int32),
        ("B", ctypes.c_int32),
        ("q_len", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("D_k", ctypes.c_int32),
        ("D_v", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("err_flags", ctypes.c_void_p),
        ("weights", ctypes.c_void_p),
        ("weights_seq_stride", ctypes.c_int64),
        ("weights_head_stride", ctypes.c_int64),
        ("weights_tokens", ctypes.c_int32),
    ]


class AppendQ4Params(ctypes.Structure):
    """Mirror of zl_kv_append_q4_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("k_new", ctypes.c_void_p),
        ("v_new", ctypes.c_void_p),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("pool", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("block_table", ctypes.c_void_p),
        ("block_table_stride", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p),
        ("new_lens", ctypes.c_void_p),
        ("B", ctypes.c_int32),
        ("q_len", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("err_flags", ctypes.c_void_p),
    ]


class ReadQ4Params(ctypes.Structure):
    """Mirror of zl_kv_read_q4_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("pool", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("block_table", ctypes.c_void_p),
        ("block_table_stride", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p),
        ("k_out", ctypes.c_void_p),
        ("v_out", ctypes.c_void_p),
        ("B", ctypes.c_int32),
        ("tokens", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("err_flags", ctypes.c_void_p),
    ]


class DecodeQ4Params(ctypes.Structure):
    """Mirror of zl_decode_attn_q4_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("q", ctypes.c_void_p),
        ("pool", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("block_table", ctypes.c_void_p),
        ("block_table_stride", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p),
        ("B", ctypes.c_int32),
        ("q_len", ctypes.c_int32),
        ("Hq", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("err_flags", ctypes.c_void_p),
        ("num_ctas", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
    ]


class NormRopeParams(ctypes.Structure):
    """Mirror of zl_qk_norm_rope_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("q_out", ctypes.c_void_p),
        ("k_out", ctypes.c_void_p),
        ("q_out_stride", ctypes.c_int64),
        ("k_out_stride", ctypes.c_int64),
        ("q_weight", ctypes.c_void_p),
        ("k_weight", ctypes.c_void_p),
        ("eps", ctypes.c_float),
        ("rope_scale", ctypes.c_float),
        ("freq_turns", ctypes.c_void_p),
        ("axes", ctypes.c_void_p),
        ("n_freq", ctypes.c_int32),
        ("n_axes", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("cache", ctypes.c_int32),
        ("positions", ctypes.c_void_p),
        ("axis_stride", ctypes.c_int64),
        ("k_pool", ctypes.c_void_p),
        ("v_pool", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("block_table", ctypes.c_void_p),
        ("block_table_stride", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p),
        ("B", ctypes.c_int32),
        ("q_len", ctypes.c_int32),
        ("Hq", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("err_flags", ctypes.c_void_p),
    ]


_lib = None
_lib_lock = threading.Lock()


def lib():
    """The loaded library (built first if missing or stale). Raises on failure."""
    global _lib
    with _lib_lock:
        if _lib is None:
            try:
                path = build()
                handle = ctypes.CDLL(path)
            except Exception as e:  # no fallback: the CUDA path is the product
                raise RuntimeError(f"libzl_decode_attn could not be built or loaded: {e}") from e
            P = ctypes.POINTER(Params)
            for name in ("zl_decode_attn", "zl_decode_attn_mla", "zl_decode_attn_noalloc"):
                fn = getattr(handle, name)
                fn.restype = ctypes.c_int
                fn.argtypes = [P, ctypes.c_void_p]
            for name in ("zl_decode_attn_workspace_size", "zl_decode_attn_mla_workspace_size"):
                fn = getattr(handle, name)
                fn.restype = ctypes.c_int
                fn.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
            handle.zl_decode_attn_launches.restype = ctypes.c_int
            handle.zl_decode_attn_launches.argtypes = [P, ctypes.POINTER(ctypes.c_int32)]
            handle.zl_kv_append.restype = ctypes.c_int
            handle.zl_kv_append.argtypes = [ctypes.POINTER(AppendParams), ctypes.c_void_p]
            S = ctypes.POINTER(ScoreParams)
            handle.zl_decode_attn_ex.restype = ctypes.c_int
            handle.zl_decode_attn_ex.argtypes = [P, S, ctypes.c_void_p]
            handle.zl_decode_attn_ex_workspace_size.restype = ctypes.c_int
            handle.zl_decode_attn_ex_workspace_size.argtypes = [P, S,
                                                                ctypes.POINTER(ctypes.c_size_t)]
            handle.zl_kv_evict.restype = ctypes.c_int
            handle.zl_kv_evict.argtypes = [ctypes.POINTER(EvictParams), ctypes.c_void_p]
            handle.zl_kv_commit.restype = ctypes.c_int
            handle.zl_kv_commit.argtypes = [ctypes.POINTER(CommitParams), ctypes.c_void_p]
            for name, mirror in (("zl_kv_append_q4", AppendQ4Params),
                                 ("zl_kv_read_q4", ReadQ4Params),
                                 ("zl_decode_attn_q4", DecodeQ4Params),
                                 ("zl_qk_norm_rope", NormRopeParams)):
                fn = getattr(handle, name)
                fn.restype = ctypes.c_int
                fn.argtypes = [ctypes.POINTER(mirror), ctypes.c_void_p]
            handle.zl_decode_attn_q4_workspace_size.restype = ctypes.c_int
            handle.zl_decode_attn_q4_workspace_size.argtypes = [ctypes.POINTER(DecodeQ4Params),
                                                                ctypes.POINTER(ctypes.c_size_t)]
            handle.zl_status_string.restype = ctypes.c_char_p
            handle.zl_status_string.argtypes = [ctypes.c_int]
            _lib = handle
        return _lib


def declared_symbols(header: str = HEADER):
    """Function names the public header declares."""
    text = open(header).read()
    return sorted(set(re.findall(r"^\s*(?:zl_status|const char\*)\s+(zl_\w+)\s*\(", text, re.M)))


def _check(status: int, what: str):
    if status != OK:
        raise ZlError(status, f"{what}: {lib().zl_status_string(status).decode()}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _pool_strides(pool: torch.Tensor, layout: str):
    """(page, token, head) element strides of a 4-D pool in NHD or HND layout."""
    if pool.dim() != 4:
        raise ValueError("pools are 4-D: [pages, slot, head, dim] (NHD) or [pages, head, slot, dim]")
    s = pool.stride()
    if layout == "NHD":
        return s[0], s[1], s[2]
    if layout == "HND":
        return s[0], s[2], s[1]
    raise ValueError(f"unknown layout {layout!r}")


def make_params(q, k_pool, v_pool, block_table, seq_lens, out, *, page_size, scale, Hkv,
                D_v, lse=None, workspace=None, err_flags=None, num_ctas=0, max_seq_len=0,
                layout="NHD", events=None, single_launch=False,
                shared_prefix_pages=0, k_new=None, v_new=None) -> Params:
    """k_new / v_new: the fused KV append (the new tokens' K and V rows, bf16
    [B, q_len, Hkv, D]; MLA: the latent rows in k_new, v_new None); the call
    then stores them in their page slots before attending."""
    B, q_len, Hq, D_qk = q.shape
    ps, ts, hs = _pool_strides(k_pool, layout)
    if v_pool is not None and _pool_strides(v_pool, layout) != (ps, ts, hs):
        raise ValueError("K and V pools must share strides")
    if k_pool.stride(3) != 1 or not q.is_contiguous() or not out.is_contiguous():
        raise ValueError("q, out and the pool rows must be contiguous")
    if block_table.stride(1) != 1:
        raise ValueError("block_table rows must be contiguous")
    p = Params()
    p.struct_size = ctypes.sizeof(Params)
    p.q, p.k_pool, p.v_pool = _ptr(q), _ptr(k_pool), _ptr(v_pool)
    p.page_stride, p.token_stride, p.head_stride = ps, ts, hs
    p.block_table = _ptr(block_table)
    p.block_table_stride = block_table.stride(0)
    p.seq_lens = _ptr(seq_lens)
    p.out, p.lse = _ptr(out), _ptr(lse)
    p.B, p.q_len, p.Hq, p.Hkv, p.D_qk, p.D_v = B, q_len, Hq, Hkv, D_qk, D_v
    p.page_size = page_size
    p.num_pages = k_pool.shape[0]
    p.max_seq_len = int(max_seq_len)
    p.scale = float(scale)
    if workspace is not None:
        p.workspace, p.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    p.err_flags = _ptr(err_flags)
    p.num_ctas = int(num_ctas)
    p.flags = SINGLE_LAUNCH if single_launch else 0
    p.shared_prefix_pages = int(shared_prefix_pages)
    for t in (k_new, v_new):
        if t is not None and not t.is_contiguous():
            raise ValueError("k_new and v_new must be contiguous")
    p.k_new, p.v_new = _ptr(k_new), _ptr(v_new)
    if events is not None:
        p.attn_begin, p.attn_end = events[0].cuda_event, events[1].cuda_event
    # The struct holds raw device pointers: keep the tensors alive with it.
    p.tensors = (q, k_pool, v_pool, block_table, seq_lens, out, lse, workspace, err_flags, events,
                 k_new, v_new)
    return p


def workspace_size(params: Params) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().zl_decode_attn_workspace_size(ctypes.byref(params), ctypes.byref(n)),
           "zl_decode_attn_workspace_size")
    return n.value


def workspace_size_mla(params: Params) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().zl_decode_attn_mla_workspace_size(ctypes.byref(params), ctypes.byref(n)),
           "zl_decode_attn_mla_workspace_size")
    return n.value


def workspace_size_ex(params: Params, scores: ScoreParams) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().zl_decode_attn_ex_workspace_size(ctypes.byref(params), ctypes.byref(scores),
                                                  ctypes.byref(n)),
           "zl_decode_attn_ex_workspace_size")
    return n.value


_ws_cache: dict = {}


def _workspace(device, nbytes, kind, counters=0):
    """A cached device byte buffer of at least nbytes per (device, kind).

    ``counters``: the call needs that many leading bytes at zero (the arrival
    counters of a single-launch GQA call). They are zeroed again whenever the
    previous user of the buffer may have written there: a call of another
    shape (its partials may sit where this call counts) or a fresh buffer.
    Calls of one shape leave the counters at zero themselves."""
    key = (device.type, device.index, kind)
    buf, last = _ws_cache.get(key, (None, None))
    if buf is None or buf.numel() < nbytes:
        buf, last = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device), None
    if counters and last != (nbytes, counters):
        buf[:counters].zero_()
    _ws_cache[key] = (buf, (nbytes, counters) if counters else None)
    return buf


def launches(params: Params) -> int:
    """Kernel launches one zl_decode_attn call with these params enqueues."""
    n = ctypes.c_int32(0)
    _check(lib().zl_decode_attn_launches(ctypes.byref(params), ctypes.byref(n)),
           "zl_decode_attn_launches")
    return int(n.value)


def call_noalloc(params: Params, stream=None):
    """zl_decode_attn_noalloc: the library's own static scratch, no workspace
    argument and no allocation (see the header for its limits)."""
    if stream is None:
        stream = torch.cuda.current_stream()
    _check(lib().zl_decode_attn_noalloc(ctypes.byref(params), ctypes.c_void_p(stream.cuda_stream)),
           "zl_decode_attn_noalloc")


def call(params: Params, *, mla: bool, stream=None):
    """Invoke the entry point on ``stream`` (default: torch's current stream)."""
    if stream is None:
        stream = torch.cuda.current_stream()
    fn = lib().zl_decode_attn_mla if mla else lib().zl_decode_attn
    _check(fn(ctypes.byref(params), ctypes.c_void_p(stream.cuda_stream)),
           "zl_decode_attn_mla" if mla else "zl_decode_attn")


def call_ex(params: Params, scores: ScoreParams, stream=None):
    """zl_decode_attn_ex on ``stream`` (default: torch's current stream)."""
    if stream is None:
        stream = torch.cuda.current_stream()
    _check(lib().zl_decode_attn_ex(ctypes.byref(params), ctypes.byref(scores),
                                   ctypes.c_void_p(stream.cuda_stream)), "zl_decode_attn_ex")


# The binding's part of a small call (a decode step of a few short sequences) is
# longer than its kernels, so the entry points below check each tensor with one
# test of all it must be, and pack the parameter structs in one step. (ctypes
# field by field, torch.cuda.current_stream() and a check per property took 37 us
# of such a call.)
_PARAMS = struct.Struct("@N3P3qPq3P9ifPNPi2PIi2P0P")
_SCORES = struct.Struct("@Nfi3P2qif0P")
_EVICT = struct.Struct("@N2P3qPqPq4P2qP2q10iPi0P")
_COMMIT = struct.Struct("@N2P3qPq2PqPP8i2P2qi0P")
_APPEND_Q4 = struct.Struct("@N2P2qP3qPq2P5iP0P")
_READ_Q4 = struct.Struct("@NP3qPq3P5iP0P")
_DECODE_Q4 = struct.Struct("@N2P3qPq3P7ifPNPiI0P")
_NORM_ROPE = struct.Struct("@N3P3q2P2q2P2f2P4iPq2P3qPqP6iP0P")
for _s, _c in ((_PARAMS, Params), (_SCORES, ScoreParams), (_EVICT, EvictParams),
               (_COMMIT, CommitParams), (_APPEND_Q4, AppendQ4Params), (_READ_Q4, ReadQ4Params),
               (_DECODE_Q4, DecodeQ4Params), (_NORM_ROPE, NormRopeParams)):
    assert _s.size == ctypes.sizeof(_c), _c.__name__


def _pack(form, *values) -> bytes:
    try:
        return form.pack(*values)
    except struct.error as e:
        raise ValueError(f"a size, count or stride is no integer, or out of range: {e}") from e


def _refuse(t, name, dtype, shape, index, contiguous):
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the K pool on device {index}")
    raise ValueError(f"{name} must be contiguous")


def _expect(t, name, dtype, shape, index, contiguous=True):
    """Check a tensor argument (index: the K pool's device, -1 the CPU); returns
    its address."""
    if (t.dtype is dtype and t.get_device() == index and t.shape == shape
            and (not contiguous or t.is_contiguous())):
        return t.data_ptr()
    return _refuse(t, name, dtype, shape, index, contiguous)


_BF16, _F32, _I32, _U32 = torch.bfloat16, torch.float32, torch.int32, torch.uint32
_U8 = torch.uint8


def _expect_cache(k_pool, v_pool, block_table, seq_lens, layout, page_size, err_flags):
    """The checks every call over a paged cache shares; returns (device index, B,
    Hkv, the pools' shape, V's width, strides in (page, token, head) order, the
    addresses of both pools, the block table and its stride, seq_lens and
    err_flags)."""
    index, shape, st = k_pool.get_device(), k_pool.shape, k_pool.stride()
    if len(shape) != 4 or (v_pool is not None and v_pool.dim() != 4):
        raise ValueError("pools are 4-D: [pages, slot, head, dim] (NHD) or "
                         "[pages, head, slot, dim] (HND)")
    if layout == "NHD":
        _, slots, Hkv, _ = shape
        ps, ts, hs, one = st
    elif layout == "HND":
        _, Hkv, slots, _ = shape
        ps, hs, ts, one = st
    else:
        raise ValueError(f"unknown layout {layout!r}")
    if k_pool.dtype is not _BF16:
        raise ValueError(f"k_pool must be {_BF16}, not {k_pool.dtype}")
    if one != 1:
        raise ValueError("pool rows must be contiguous")
    v_at = width_v = 0
    if v_pool is not None:
        width_v = v_pool.shape[3]
        v_at = _expect(v_pool, "v_pool", _BF16, (*shape[:3], width_v), index, False)
        if v_pool.stride() != st:
            raise ValueError("K and V pools must share strides, and their rows be contiguous")
    if slots != page_size:
        raise ValueError(f"the pools hold {slots} slots per page, page_size is {page_size}")
    if block_table.dim() != 2:
        raise ValueError("block_table must be 2-D")
    B, width = block_table.shape
    sl_at = _expect(seq_lens, "seq_lens", _I32, (B,), index)
    bt_stride, one = block_table.stride()
    if B == 1:
        bt_stride = width
    if (block_table.dtype is not _I32 or block_table.get_device() != index or one != 1
            or bt_stride < width):
        _expect(block_table, "block_table", _I32, (B, width), index)
        raise ValueError("block_table rows must be contiguous and distinct")
    err = 0
    if err_flags is not None:
        if err_flags.dtype is not _I32 and err_flags.dtype is not _U32 or err_flags.numel() < 1:
            raise ValueError("err_flags must be a 32-bit integer tensor")
        if err_flags.get_device() != index:
            raise ValueError(f"err_flags is on {err_flags.device}, the K pool on device {index}")
        err = err_flags.data_ptr()
    return (index, B, Hkv, shape, width_v, ps, ts, hs, k_pool.data_ptr(), v_at,
            block_table.data_ptr(), bt_stride, sl_at, err)


def _token_rows(t, name, B, Hkv, index):
    """fp32 [B, Hkv, tokens] with contiguous token rows; returns (address,
    sequence stride, head stride, tokens)."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [B, Hkv, tokens]")
    n = t.shape[2]
    at = _expect(t, name, _F32, (B, Hkv, n), index, False)
    seq, head, one = t.stride()
    if n < 1 or (n > 1 and one != 1):
        raise ValueError(f"{name} needs contiguous rows of at least one token")
    return at, seq, head, n


def _on(index, stream):
    """The raw stream a call goes to (the device's current one by default), and
    the context its scratch is allocated in: memory from torch's allocator is
    reused in the order of that stream."""
    if index < 0:
        raise ValueError("the tensors are not on a CUDA device")
    if index != torch._C._cuda_getDevice():
        raise ValueError(f"the pools are on CUDA device {index}, which is not the current one")
    cur = torch._C._cuda_getCurrentRawStream(index)
    if stream is None or stream.cuda_stream == cur:
        return cur, _NO_CONTEXT
    return stream.cuda_stream, torch.cuda.stream(stream)


_NO_CONTEXT = contextlib.nullcontext()
_raw: dict = {}
_sizes: dict = {}  # workspace bytes of zl_decode_attn_ex by device and shapes


def _raw_fn(name, nargs):
    """The entry point taking packed structs (bytes) and plain addresses."""
    fn = _raw.get(name)
    if fn is None:
        fn = lib()[name]  # a function object of its own: lib().name keeps its types
        fn.restype = ctypes.c_int
        fn.argtypes = [ctypes.c_char_p] * nargs + [ctypes.c_void_p]
        _raw[name] = fn
    return fn


def make_score_params(q, Hkv, *, softcap=0.0, alibi_slopes=None, window=0, tree_mask=None,
                      weights=None, weights_decay=1.0) -> ScoreParams:
    """The score modifications of a decode_attn call (see there), for call_ex."""
    m = ScoreParams.from_buffer_copy(_pack_scores(
        *q.shape[:3], Hkv, q.get_device(), softcap, alibi_slopes, window, tree_mask, weights,
        weights_decay)[0])
    m.tensors = (alibi_slopes, tree_mask, weights)
    return m


def _pack_scores(B, q_len, Hq, Hkv, index, softcap, alibi_slopes, window, tree_mask, weights,
                 weights_decay):
    """zl_score_params as bytes, and the length of the weights rows (0: none)."""
    slopes = mask = w = ws = wh = wt = 0
    if alibi_slopes is not None:
        slopes = _expect(alibi_slopes, "alibi_slopes", _F32, (Hq,), index)
    if tree_mask is not None:
        if tree_mask.dtype is not _I32 and tree_mask.dtype is not _U32:
            raise ValueError("tree_mask must be 32-bit words")
        mask = _expect(tree_mask, "tree_mask", tree_mask.dtype, (B, q_len, (q_len + 31) // 32),
                       index)
    if weights is not None:
        w, ws, wh, wt = _token_rows(weights, "weights", B, Hkv, index)
    return _pack(_SCORES, _SCORES.size, softcap, window, slopes, mask, w, ws, wh, wt,
                 weights_decay), wt


def _run_ex(q, k_pool, v_pool, block_table, seq_lens, page_size, scale, out, lse, workspace,
            err_flags, num_ctas, max_seq_len, layout, stream, events, k_new, v_new, softcap,
            alibi_slopes, window, tree_mask, weights, weights_decay):
    """decode_attn with modified scores (zl_decode_attn_ex)."""
    if q.dim() != 4 or v_pool is None:
        raise ValueError("q must be [B, q_len, Hq, D], with K and V pools")
    (index, B, Hkv, pool_shape, width_v, ps, ts, hs, k_at, v_at, bt_at, bt_stride, sl_at,
     err) = _expect_cache(k_pool, v_pool, block_table, seq_lens, layout, page_size, err_flags)
    shape = q.shape
    _, q_len, Hq, D = shape
    if width_v != D:
        raise ValueError("q and the pools' rows must be equally wide")
    q_at = _expect(q, "q", _BF16, (B, q_len, Hq, pool_shape[3]), index)
    out_at = lse_at = kn = vn = begin = end = 0
    if out is not None:
        out_at = _expect(out, "out", _BF16, shape, index)
    if lse is not None:
        lse_at = _expect(lse, "lse", _F32, (B, q_len, Hq), index)
    if k_new is not None:
        kn = _expect(k_new, "k_new", _BF16, (B, q_len, Hkv, D), index)
    if v_new is not None:
        vn = _expect(v_new, "v_new", _BF16, (B, q_len, Hkv, D), index)
    mods, tokens = _pack_scores(B, q_len, Hq, Hkv, index, softcap, alibi_slopes, window,
                                tree_mask, weights, weights_decay)
    if events is not None:
        begin, end = events[0].cuda_event or 0, events[1].cuda_event or 0
    on, scratch = _on(index, stream)

    def params(out_at, ws_at, ws_bytes):
        return _pack(
            _PARAMS, _PARAMS.size, q_at, k_at, v_at, ps, ts, hs, bt_at, bt_stride, sl_at, out_at,
            lse_at, B, q_len, Hq, Hkv, D, D, page_size, pool_shape[0], max_seq_len, scale, ws_at,
            ws_bytes, err, num_ctas, begin, end, 0, 0, kn, vn)

    with scratch:
        if out is None:
            out = torch.empty(shape, dtype=_BF16, device=q.device)
            out_at = out.data_ptr()
        if workspace is None:
            # a call's own: stream order alone separates it from other calls,
            # and a captured graph keeps it. Its size follows from the shapes.
            key = (index, B, q_len, Hq, Hkv, page_size, bt_stride, num_ctas, max_seq_len, window,
                   tokens)
            ws_bytes = _sizes.get(key)
            if ws_bytes is None:
                n = ctypes.c_size_t(0)
                _check(_raw_fn("zl_decode_attn_ex_workspace_size", 2)(
                    params(out_at, 0, 0), mods, ctypes.addressof(n)),
                    "zl_decode_attn_ex_workspace_size")
                if len(_sizes) >= 4096:
                    _sizes.clear()
                ws_bytes = _sizes[key] = n.value or 256
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
        else:
            ws_bytes = workspace.numel() * workspace.element_size()
        status = _raw_fn("zl_decode_attn_ex", 2)(
            params(out_at, workspace.data_ptr(), ws_bytes), mods, on)
        if status != OK:
            _check(status, "zl_decode_attn_ex")
    return out


def _run(q, k_pool, v_pool, block_table, seq_lens, *, mla, page_size, scale, Hkv, D_v, out, lse,
         workspace, err_flags, num_ctas, max_seq_len, layout, stream, events, single_launch=False,
         shared_prefix_pages=0, k_new=None, v_new=None):
    if out is None:
        out = torch.empty(q.shape[:3] + (D_v,), dtype=torch.bfloat16, device=q.device)
    p = make_params(q, k_pool, v_pool, block_table, seq_lens, out, page_size=page_size,
                    scale=scale, Hkv=Hkv, D_v=D_v, lse=lse, err_flags=err_flags,
                    num_ctas=num_ctas, max_seq_len=max_seq_len, layout=layout, events=events,
                    single_launch=single_launch, shared_prefix_pages=shared_prefix_pages,
                    k_new=k_new, v_new=v_new)
    need = workspace_size_mla(p) if mla else workspace_size(p)
    if workspace is None:
        counters = 8 * q.shape[0] * Hkv if single_launch else 0
        workspace = _workspace(q.device, need,
                               "mla" if mla else ("gqa1" if single_launch else "gqa"), counters)
    p.workspace = workspace.data_ptr()
    p.workspace_bytes = workspace.numel() * workspace.element_size()
    call(p, mla=mla, stream=stream)
    return out


def decode_attn(q, k_pool, v_pool, block_table, seq_lens, *, page_size, scale, out=None, lse=None,
                workspace=None, err_flags=None, num_ctas=0, max_seq_len=0, layout="NHD",
                stream=None, events=None, single_launch=False, shared_prefix_pages=0,
                k_new=None, v_new=None, softcap=0.0, alibi_slopes=None, window=0, tree_mask=None,
                weights=None, weights_decay=1.0):
    """GQA/MHA/MQA paged decode attention (zl_decode_attn).

    q [B, q_len, Hq, 128] bf16; k_pool, v_pool [pages, page_size, Hkv, 128]
    (layout "NHD") or [pages, Hkv, page_size, 128] ("HND") bf16; block_table
    int32 [B, max_pages]; seq_lens int32 [B]. Returns out [B, q_len, Hq, 128]
    bf16. single_launch: merge split-KV partials inside the attention kernel
    (ZL_DECODE_SINGLE_LAUNCH; a caller's workspace must then hold zeroed
    arrival counters, see the header; the default cached one is kept so).
    shared_prefix_pages: the first pages of every block-table row are the same
    shared prefix (read once per group of sequences; see the header).
    k_new, v_new: the q_len new tokens' K and V rows [B, q_len, Hkv, 128] bf16;
    the call stores them in their page slots (as kv_append does) and then
    attends, in the same launch.

    Modified scores (zl_decode_attn_ex; not with single_launch or
    shared_prefix_pages), for query position pos and token position t:
    softcap: s -> softcap * tanh(s / softcap). alibi_slopes [Hq] fp32: s ->
    s - slope * (pos - t). window: tokens with pos - t < window are seen.
    tree_mask int32 [B, q_len, ceil(q_len / 32)]: the q_len query tokens are a
    drafted tree, bit j of row i set where token i sees drafted token j (see
    tree_mask()). weights fp32 [B, Hkv, tokens]: each cached token's softmax
    weight, summed over the query tokens and the heads of its kv head, is added
    to weights_decay times what it holds. A new token's sum starts from what its
    element held, so keep the elements behind seq_lens at 0. The scratch of such
    a call grows with the rows' length (4 bytes per query row and token): give
    wide rows as weights[:, :, :n], n of at least the longest sequence.
    """
    if (softcap or window or alibi_slopes is not None or tree_mask is not None
            or weights is not None):
        if single_launch or shared_prefix_pages:
            raise ZlError(ERR_UNSUPPORTED, "modified scores with single_launch or a shared prefix")
        return _run_ex(q, k_pool, v_pool, block_table, seq_lens, page_size, scale, out, lse,
                       workspace, err_flags, num_ctas, max_seq_len, layout, stream, events, k_new,
                       v_new, softcap, alibi_slopes, window, tree_mask, weights, weights_decay)
    Hkv = k_pool.shape[2] if layout == "NHD" else k_pool.shape[1]
    return _run(q, k_pool, v_pool, block_table, seq_lens, mla=False, page_size=page_size,
                scale=scale, Hkv=Hkv, D_v=q.shape[3], out=out, lse=lse, workspace=workspace,
                err_flags=err_flags, num_ctas=num_ctas, max_seq_len=max_seq_len, layout=layout,
                stream=stream, events=events, single_launch=single_launch,
                shared_prefix_pages=shared_prefix_pages, k_new=k_new, v_new=v_new)


def decode_attn_mla(q, kv_pool, block_table, seq_lens, *, page_size, scale, D_v=512, out=None,
                    lse=None, workspace=None, err_flags=None, num_ctas=0, max_seq_len=0,
                    stream=None, events=None, kv_new=None):
    """Absorbed MLA paged decode (zl_decode_attn_mla).

    q [B, q_len, Hq, 576] bf16; kv_pool [pages, page_size, 1, 576] bf16 (V =
    first D_v columns). Returns out [B, q_len, Hq, D_v] bf16. kv_new: the new
    tokens' latent rows [B, q_len, 1, 576] bf16, stored in their page slots by
    the same launch before it attends.
    """
    return _run(q, kv_pool, None, block_table, seq_lens, mla=True, page_size=page_size,
                scale=scale, Hkv=1, D_v=D_v, out=out, lse=lse, workspace=workspace,
                err_flags=err_flags, num_ctas=num_ctas, max_seq_len=max_seq_len, layout="NHD",
                stream=stream, events=events, k_new=kv_new)


def make_append_params(k_new, v_new, k_pool, v_pool, block_table, seq_lens, *, page_size,
                       layout="NHD", err_flags=None) -> AppendParams:
    B, q_len, Hkv, D_k = k_new.shape
    ps, ts, hs = _pool_strides(k_pool, layout)
    if (v_pool is None) != (v_new is None):
        raise ValueError("v_new and v_pool are given together (both None for a latent-only pool)")
    if v_pool is not None and _pool_strides(v_pool, layout) != (ps, ts, hs):
        raise ValueError("K and V pools must share strides")
    if not k_new.is_contiguous() or (v_new is not None and not v_new.is_contiguous()):
        raise ValueError("k_new and v_new must be contiguous")
    if k_pool.stride(3) != 1 or block_table.stride(1) != 1:
        raise ValueError("pool rows and block_table rows must be contiguous")
    p = AppendParams()
    p.struct_size = ctypes.sizeof(AppendParams)
    p.k_new, p.v_new, p.k_pool, p.v_pool = _ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool)
    p.page_stride, p.token_stride, p.head_stride = ps, ts, hs
    p.block_table = _ptr(block_table)
    p.block_table_stride = block_table.stride(0)
    p.seq_lens = _ptr(seq_lens)
    p.B, p.q_len, p.Hkv, p.D_k = B, q_len, Hkv, D_k
    p.D_v = 0 if v_new is None else v_new.shape[3]
    p.page_size = page_size
    p.num_pages = k_pool.shape[0]
    p.err_flags = _ptr(err_flags)
    p.tensors = (k_new, v_new, k_pool, v_pool, block_table, seq_lens, err_flags)
    return p


def kv_append(k_new, v_new, k_pool, v_pool, block_table, seq_lens, *, page_size, layout="NHD",
              err_flags=None, stream=None):
    """Paged KV append (zl_kv_append): new token i of sequence b goes to logical
    position seq_lens[b] - q_len + i of its cache, in place.

    k_new [B, q_len, Hkv, D_k] bf16, v_new [B, q_len, Hkv, D_v] bf16 or None
    (latent-only pool, v_pool None); pools, block_table and seq_lens as for
    decode_attn (seq_lens count the new tokens).
    """
    p = make_append_params(k_new, v_new, k_pool, v_pool, block_table, seq_lens,
                           page_size=page_size, layout=layout, err_flags=err_flags)
    if stream is None:
        stream = torch.cuda.current_stream()
    _check(lib().zl_kv_append(ctypes.byref(p), ctypes.c_void_p(stream.cuda_stream)),
           "zl_kv_append")


def tree_mask(parents) -> torch.Tensor:
    """The ancestor bits decode_attn's tree_mask takes, from drafted trees.

    parents: int [B, q_len] on the host (list, array or CPU tensor): the index
    of each drafted token's parent, smaller than its own, or -1 for a child of
    the context's last token. Host-side planning, as for a block table; returns
    int32 [B, q_len, ceil(q_len / 32)] on the CPU.
    """
    par = torch.as_tensor(parents)
    if par.dim() != 2 or par.is_floating_point() or par.is_cuda:
        raise ValueError("parents must be int [B, q_len] on the host")
    par = par.to(torch.int64)
    B, q_len = par.shape
    if ((par < -1) | (par >= torch.arange(q_len))).any():
        raise ValueError("a parent's index is -1 or smaller than its child's")
    words = torch.zeros(B, q_len, (q_len + 31) // 32, dtype=torch.int64)
    rows = torch.arange(B)
    for i in range(q_len):
        p = par[:, i]
        words[:, i] = torch.where(p[:, None] >= 0, words[rows, p.clamp(min=0)], 0)
        words[:, i, i // 32] |= 1 << (i % 32)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def kv_evict(k_pool, v_pool, block_table, seq_lens, weights, *, page_size, budget, sink=0,
             recent=0, new_lens=None, kept=None, weights_out=None, dst_block_table=None,
             clear_weights=False, layout="NHD", err_flags=None, stream=None):
    """Hold every (sequence, kv head) to ``budget`` cached tokens (zl_kv_evict).

    weights [B, Hkv, tokens] fp32, as decode_attn accumulates them: a sequence
    of more than budget tokens keeps its first ``sink``, its last ``recent``
    and the ones between with the largest weights, in order; their K, V and
    weights move to the front. In place, or to the pages of dst_block_table
    (weights to weights_out when given). v_pool None: a latent-only pool.
    clear_weights: the weights behind the new length, which belong to no token
    any more, become 0 (in place up to the old length, in weights_out up to the
    end of its rows); otherwise they stay, and the next tokens cached there
    start from them. Rows much wider than the sequences take longer to search:
    give weights[:, :, :n] here too. Returns (new_lens int32 [B], kept int32
    [B, Hkv, budget]: the kept positions, then -1).
    """
    if weights is None:
        raise ValueError("weights is required")
    (index, B, Hkv, shape, width_v, ps, ts, hs, k_at, v_at, bt_at, bt_stride, sl_at,
     err) = _expect_cache(k_pool, v_pool, block_table, seq_lens, layout, page_size, err_flags)
    w, w_seq, w_head, tokens = _token_rows(weights, "weights", B, Hkv, index)
    wo = wo_seq = wo_head = dst = dst_stride = 0
    clear = tokens if clear_weights else 0
    if weights_out is not None:
        wo, wo_seq, wo_head, out_tokens = _token_rows(weights_out, "weights_out", B, Hkv, index)
        if out_tokens < min(budget, tokens):
            raise ValueError("weights_out is shorter than what the budget may leave")
        clear = out_tokens if clear_weights else 0
    if dst_block_table is not None:
        if dst_block_table.dim() != 2:
            raise ValueError("dst_block_table must be 2-D")
        width = dst_block_table.shape[1]
        dst = _expect(dst_block_table, "dst_block_table", _I32, (B, width), index, False)
        dst_stride, one = dst_block_table.stride()
        if B == 1:
            dst_stride = width
        if one != 1 or dst_stride < width:
            raise ValueError("dst_block_table rows must be contiguous and distinct")
    new_at = kept_at = 0
    if new_lens is not None:
        new_at = _expect(new_lens, "new_lens", _I32, (B,), index)
    if kept is not None:
        kept_at = _expect(kept, "kept", _I32, (B, Hkv, budget), index)
    on, scratch = _on(index, stream)
    if new_lens is None or kept is None:
        with scratch:
            if new_lens is None:
                new_lens = torch.empty(B, dtype=_I32, device=k_pool.device)
                new_at = new_lens.data_ptr()
            if kept is None:
                kept = torch.empty(B, Hkv, max(budget, 1), dtype=_I32, device=k_pool.device)
                kept_at = kept.data_ptr()
    status = _raw_fn("zl_kv_evict", 1)(_pack(
        _EVICT, _EVICT.size, k_at, v_at, ps, ts, hs, bt_at, bt_stride, dst, dst_stride, sl_at,
        new_at, kept_at, w, w_seq, w_head, wo, wo_seq, wo_head, tokens, B, Hkv, shape[3], width_v,
        page_size, shape[0], budget, sink, recent, err, clear), on)
    if status != OK:
        _check(status, "zl_kv_evict")
    return new_lens, kept


def kv_commit(k_pool, v_pool, block_table, seq_lens, path, accepted, *, page_size, q_len,
              new_lens=None, weights=None, layout="NHD", err_flags=None, stream=None):
    """Move the accepted path of a drafted tree behind the context (zl_kv_commit).

    The last q_len of each sequence's seq_lens[b] tokens are the drafted tree;
    its tokens path[b, :accepted[b]] (path int32 [B, n], accepted int32 [B])
    become the tokens after the context, in place. v_pool None: a latent-only
    pool. weights [B, Hkv, tokens] fp32, as decode_attn accumulates them: the
    accepted tokens' sums move with them, the rejected ones' become 0 (without
    it they stay where the drafted tokens were). Returns new_lens int32 [B]
    (context plus accepted).
    """
    (index, B, Hkv, shape, width_v, ps, ts, hs, k_at, v_at, bt_at, bt_stride, sl_at,
     err) = _expect_cache(k_pool, v_pool, block_table, seq_lens, layout, page_size, err_flags)
    if path.dim() != 2:
        raise ValueError("path must be 2-D")
    n = path.shape[1]
    path_at = _expect(path, "path", _I32, (B, n), index, False)
    path_stride, one = path.stride()
    if n > 1 and one != 1:
        raise ValueError("path rows must be contiguous")
    acc = _expect(accepted, "accepted", _I32, (B,), index)
    w = w_seq = w_head = tokens = 0
    if weights is not None:
        w, w_seq, w_head, tokens = _token_rows(weights, "weights", B, Hkv, index)
    new_at = 0
    if new_lens is not None:
        new_at = _expect(new_lens, "new_lens", _I32, (B,), index)
    on, scratch = _on(index, stream)
    if new_lens is None:
        with scratch:
            new_lens = torch.empty(B, dtype=_I32, device=k_pool.device)
            new_at = new_lens.data_ptr()
    status = _raw_fn("zl_kv_commit", 1)(_pack(
        _COMMIT, _COMMIT.size, k_at, v_at, ps, ts, hs, bt_at, bt_stride, sl_at, path_at,
        path_stride if B > 1 else n, acc, new_at, n, B, q_len, Hkv, shape[3], width_v, page_size,
        shape[0], err, w, w_seq, w_head, tokens), on)
    if status != OK:
        _check(status, "zl_kv_commit")
    return new_lens


# ------------------------------------------------------------- a cache in 4 bits
def _pool_layout(shape, st, layout):
    """(slots, heads, page stride, token stride, head stride) of a 4-D pool."""
    if len(shape) != 4:
        raise ValueError("pools are 4-D: [pages, slot, head, dim] (NHD) or "
                         "[pages, head, slot, dim] (HND)")
    if st[3] != 1:
        raise ValueError("pool rows must be contiguous")
    if layout == "NHD":
        return shape[1], shape[2], st[0], st[1], st[2]
    if layout == "HND":
        return shape[2], shape[1], st[0], st[2], st[1]
    raise ValueError(f"unknown layout {layout!r}")


def _expect_table(block_table, seq_lens, index, err_flags):
    """Block table, lengths and error word; returns (B, addresses of the table, its
    stride, of seq_lens and err_flags)."""
    shape = block_table.shape
    if len(shape) != 2:
        raise ValueError("block_table must be 2-D")
    B, bt_stride = shape
    if (block_table.dtype is not _I32 or block_table.get_device() != index
            or not block_table.is_contiguous()):
        _expect(block_table, "block_table", _I32, shape, index, False)
        width, st = bt_stride, block_table.stride()
        bt_stride = st[0] if B > 1 else width
        if (width > 1 and st[1] != 1) or bt_stride < width:
            raise ValueError("block_table rows must be contiguous and distinct")
    if (seq_lens.dtype is not _I32 or seq_lens.get_device() != index or seq_lens.shape != (B,)
            or not seq_lens.is_contiguous()):
        _refuse(seq_lens, "seq_lens", _I32, (B,), index, True)
    err = 0
    if err_flags is not None:
        if err_flags.dtype is not _I32 and err_flags.dtype is not _U32 or err_flags.numel() < 1:
            raise ValueError("err_flags must be a 32-bit integer tensor")
        if err_flags.get_device() != index:
            raise ValueError(f"err_flags is on {err_flags.device}, the pool on device {index}")
        err = err_flags.data_ptr()
    return B, block_table.data_ptr(), bt_stride, seq_lens.data_ptr(), err


def _expect_q4(pool, block_table, seq_lens, layout, page_size, err_flags):
    """The checks every call over a 4-bit cache shares; returns (device index, B, Hkv,
    num_pages, address, strides in (page, token, head) order, then the block table,
    its stride, seq_lens and err_flags)."""
    index, shape, st = pool.get_device(), pool.shape, pool.stride()
    if pool.dtype is not _U8 or len(shape) != 4 or shape[3] != Q4_ROW_BYTES:
        raise ValueError(f"the pool must be uint8 with rows of {Q4_ROW_BYTES} bytes: "
                         "[pages, slot, head, row] (NHD) or [pages, head, slot, row] (HND)")
    slots, Hkv, ps, ts, hs = _pool_layout(shape, st, layout)
    if slots != page_size:
        raise ValueError(f"the pool holds {slots} slots per page, page_size is {page_size}")
    B, bt_at, bt_stride, sl_at, err = _expect_table(block_table, seq_lens, index, err_flags)
    return (index, B, Hkv, shape[0], pool.data_ptr(), ps, ts, hs, bt_at, bt_stride, sl_at, err)


def _expect_rows(t, name, shape, B, q_len, heads, index):
    """bf16 [B, q_len, heads, 128] (shape: the tensor's own) whose heads lie side by side
    and whose tokens are evenly spaced (a slice of a fused projection's output is); returns
    (address, token stride)."""
    if t.dtype is not _BF16 or t.get_device() != index or shape != (B, q_len, heads, 128):
        _refuse(t, name, _BF16, (B, q_len, heads, 128), index, False)
    if t.is_contiguous():
        return t.data_ptr(), heads * 128
    sb, st, sh, one = t.stride()
    if one != 1 or (heads > 1 and sh != 128):
        raise ValueError(f"{name}: the heads of a token must lie side by side")
    if q_len == 1:
        st = sb if B > 1 else heads * 128
    elif B > 1 and sb != q_len * st:
        raise ValueError(f"{name}: the tokens must be evenly spaced across the batch")
    return t.data_ptr(), st


def kv_append_q4(k_new, v_new, pool, block_table, seq_lens, *, page_size, new_lens=None,
                 layout="NHD", err_flags=None, stream=None):
    """Store new tokens' K and V rows in a 4-bit cache, quantised (zl_kv_append_q4).

    k_new, v_new [B, q_len, Hkv, 128] bf16 (slices of a fused projection's output are
    taken as they are); pool uint8 [pages, page_size, Hkv, 144] (layout "NHD") or
    [pages, Hkv, page_size, 144] ("HND"); block_table and seq_lens as for kv_append
    (seq_lens count the new tokens). new_lens int32 [B]: a padded batch; sequence b's
    new tokens are its first new_lens[b] rows.
    """
    (index, B, Hkv, pages, at, ps, ts, hs, bt_at, bt_stride, sl_at,
     err) = _expect_q4(pool, block_table, seq_lens, layout, page_size, err_flags)
    shape = k_new.shape
    if len(shape) != 4:
        raise ValueError("k_new must be [B, q_len, Hkv, 128]")
    q_len = shape[1]
    k_at, k_st = _expect_rows(k_new, "k_new", shape, B, q_len, Hkv, index)
    v_at, v_st = _expect_rows(v_new, "v_new", v_new.shape, B, q_len, Hkv, index)
    n_at = 0
    if new_lens is not None:
        n_at = _expect(new_lens, "new_lens", _I32, (B,), index)
    on, _ = _on(index, stream)
    status = (_raw.get("zl_kv_append_q4") or _raw_fn("zl_kv_append_q4", 1))(_pack(
        _APPEND_Q4, _APPEND_Q4.size, k_at, v_at, k_st, v_st, at, ps, ts, hs, bt_at, bt_stride,
        sl_at, n_at, B, q_len, Hkv, page_size, pages, err), on)
    if status != OK:
        _check(status, "zl_kv_append_q4")


def kv_read_q4(pool, block_table, seq_lens, *, page_size, tokens=None, k_out=None, v_out=None,
               layout="NHD", err_flags=None, stream=None):
    """Read a 4-bit cache's tokens back as bf16 (zl_kv_read_q4).

    Writes rows t < seq_lens[b] of k_out and v_out [B, tokens, Hkv, 128] bf16 (exactly
    the values the codes stand for) and leaves the rows behind them as they are; tokens
    must hold the longest sequence. Without k_out and v_out, both are made (zeros behind
    the lengths) for the given ``tokens``; with one of them, only that is written.
    Returns (k_out, v_out).
    """
    (index, B, Hkv, pages, at, ps, ts, hs, bt_at, bt_stride, sl_at,
     err) = _expect_q4(pool, block_table, seq_lens, layout, page_size, err_flags)
    given = k_out if k_out is not None else v_out
    if given is not None:
        shape = given.shape
        if len(shape) != 4:
            raise ValueError("k_out and v_out must be [B, tokens, Hkv, 128]")
        if tokens is not None and tokens != shape[1]:
            raise ValueError(f"tokens is {tokens}, the outputs hold {shape[1]}")
        tokens = shape[1]
    elif tokens is None or tokens < 1:
        raise ValueError("tokens (at least the longest sequence) or the outputs are required")
    on, scratch = _on(index, stream)
    if given is None:
        with scratch:
            k_out = torch.zeros(B, tokens, Hkv, 128, dtype=_BF16, device=pool.device)
            v_out = torch.zeros_like(k_out)
    k_at = v_at = 0
    if k_out is not None:
        k_at = _expect(k_out, "k_out", _BF16, (B, tokens, Hkv, 128), index)
    if v_out is not None:
        v_at = _expect(v_out, "v_out", _BF16, (B, tokens, Hkv, 128), index)
    status = (_raw.get("zl_kv_read_q4") or _raw_fn("zl_kv_read_q4", 1))(_pack(
        _READ_Q4, _READ_Q4.size, at, ps, ts, hs, bt_at, bt_stride, sl_at, k_at, v_at, B, tokens,
        Hkv, page_size, pages, err), on)
    if status != OK:
        _check(status, "zl_kv_read_q4")
    return k_out, v_out


def decode_attn_q4(q, pool, block_table, seq_lens, *, page_size, scale, out=None, lse=None,
                   workspace=None, err_flags=None, num_ctas=0, max_seq_len=0, layout="NHD",
                   stream=None):
    """Paged decode attention over a 4-bit cache (zl_decode_attn_q4).

    q [B, q_len, Hq, 128] bf16; pool uint8 [pages, page_size, Hkv, 144] (layout "NHD") or
    [pages, Hkv, page_size, 144] ("HND"), as kv_append_q4 or qk_norm_rope fill it;
    block_table int32 [B, max_pages], seq_lens int32 [B]: as for decode_attn, the q_len
    query tokens being the last cached ones. Returns out [B, q_len, Hq, 128] bf16; lse
    fp32 [B, q_len, Hq] is written when given.
    """
    (index, B, Hkv, pages, at, ps, ts, hs, bt_at, bt_stride, sl_at,
     err) = _expect_q4(pool, block_table, seq_lens, layout, page_size, err_flags)
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [B, q_len, Hq, 128]")
    _, q_len, Hq, _ = shape
    if (shape != (B, q_len, Hq, 128) or q.dtype is not _BF16 or q.get_device() != index
            or not q.is_contiguous()):
        _refuse(q, "q", _BF16, (B, q_len, Hq, 128), index, True)
    q_at = q.data_ptr()
    out_at = lse_at = 0
    if out is not None:
        out_at = _expect(out, "out", _BF16, shape, index)
    if lse is not None:
        lse_at = _expect(lse, "lse", _F32, (B, q_len, Hq), index)
    on, scratch = _on(index, stream)
    if workspace is None:
        key = ("q4", index, B, q_len, Hq, Hkv, page_size, bt_stride, num_ctas, max_seq_len)
        ws_bytes = _sizes.get(key)
        if ws_bytes is None:
            n = ctypes.c_size_t(0)
            _check(_raw_fn("zl_decode_attn_q4_workspace_size", 1)(_pack(
                _DECODE_Q4, _DECODE_Q4.size, q_at, at, ps, ts, hs, bt_at, bt_stride, sl_at, out_at,
                lse_at, B, q_len, Hq, Hkv, page_size, pages, max_seq_len, scale, 0, 0, err,
                num_ctas, 0), ctypes.addressof(n)), "zl_decode_attn_q4_workspace_size")
            if len(_sizes) >= 4096:
                _sizes.clear()
            ws_bytes = _sizes[key] = n.value
    else:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous and on the pool's device")
        ws_bytes = workspace.numel() * workspace.element_size()
    if out is None or (workspace is None and ws_bytes):
        with scratch:
            if out is None:
                out = torch.empty(shape, dtype=_BF16, device=q.device)
                out_at = out.data_ptr()
            if workspace is None and ws_bytes:  # a call's own, as in _run_ex
                workspace = torch.empty(ws_bytes, dtype=_U8, device=q.device)
    status = (_raw.get("zl_decode_attn_q4") or _raw_fn("zl_decode_attn_q4", 1))(_pack(
        _DECODE_Q4, _DECODE_Q4.size, q_at, at, ps, ts, hs, bt_at, bt_stride, sl_at, out_at, lse_at,
        B, q_len, Hq, Hkv, page_size, pages, max_seq_len, scale,
        0 if workspace is None else workspace.data_ptr(), ws_bytes, err, num_ctas, 0), on)
    if status != OK:
        _check(status, "zl_decode_attn_q4")
    return out


def rope_frequencies(dim=128, base=10000.0):
    """The usual rotation frequencies of ``dim`` rotated elements, in radians per
    position: base^(-2 i / dim), i < dim / 2 (a list of floats, for Rope)."""
    return [float(base) ** (-2.0 * i / dim) for i in range(dim // 2)]


class Rope:
    """A rotation by position, laid out once for qk_norm_rope.

    frequencies: radians per position of each rotated pair (numbers in 64 bits on the
    host; 16, 32, 48 or 64 of them: twice as many elements of a head are rotated, the
    first ones), scaled as a model wants them. axes: which row of the positions each
    follows (default: all the first). interleaved: pairs are (2 i, 2 i + 1) instead of
    (i, n + i). scale: factor of the rotated elements.
    """

    def __init__(self, frequencies, *, axes=None, interleaved=False, scale=1.0):
        freq = [float(f) for f in frequencies]
        axes = [0] * len(freq) if axes is None else [int(a) for a in axes]
        if len(axes) != len(freq):
            raise ValueError("axes must name one axis for every frequency")
        if any(not math.isfinite(f) for f in freq) or any(not 0 <= a < 4 for a in axes):
            raise ValueError("frequencies must be finite, axes 0 to 3")
        self.n_freq, self.interleaved, self.scale = len(freq), bool(interleaved), float(scale)
        self.n_axes = max(axes, default=0) + 1
        # turns per position, 64 bits behind the point: f / (2 pi) in whole numbers, as
        # a float's quotient would not hold the digits that position * turns needs
        turns = []
        for f in freq:
            num, den = f.as_integer_ratio()
            turns.append((2 * num * _INV_TWO_PI + (den << 192)) // (den << 193) % (1 << 64))
        self._lay_out(turns, axes)

    def _lay_out(self, turns, axes):
        self._turns = (ctypes.c_uint64 * max(1, len(turns)))(*turns)
        self._axes = (ctypes.c_uint8 * max(1, len(axes)))(*axes)

    # Copies and pickles carry the numbers and lay out arrays of their own (a call takes the
    # arrays' addresses, so none is kept here that could outlive them).
    def __getstate__(self):
        return {**self.__dict__, "_turns": list(self._turns), "_axes": list(self._axes)}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._lay_out(state["_turns"], state["_axes"])


# 2^256 / (2 pi), from pi to 80 digits
_INV_TWO_PI = ((10 ** 80 << 255)
               // 314159265358979323846264338327950288419716939937510582097494459230781640628620899)
_NO_ROPE = Rope([])


def qk_norm_rope(q, k, *, rope=None, positions=None, q_weight=None, k_weight=None, eps=1e-6,
                 q_out=None, k_out=None, v=None, k_pool=None, v_pool=None, pool=None,
                 block_table=None, seq_lens=None, page_size=0, layout="NHD", err_flags=None,
                 stream=None):
    """Norm and rotation of queries and keys per head, in one pass (zl_qk_norm_rope).

    q [B, q_len, Hq, 128], k [B, q_len, Hkv, 128] bf16 (slices of a fused projection's
    output are taken as they are). q_weight, k_weight fp32 [128]: RMS norm over each head
    with eps; None: no norm. rope (Rope): the rotation, None: none. positions int32
    [B, q_len], or [axes, B, q_len] for a rope of several axes; None: the tokens' places
    in the cache, seq_lens[b] - q_len + i. q_out and k_out may be q and k themselves.

    With a cache the keys and the rows of v [B, q_len, Hkv, 128] also go to their page
    slots: bf16 pools k_pool, v_pool as kv_append would store them, or the 4-bit ``pool``
    as kv_append_q4 would. k_out is then written only when given. Returns (q_out, k_out).
    """
    q_shape, k_shape = q.shape, k.shape
    if len(q_shape) != 4 or len(k_shape) != 4:
        raise ValueError("q and k must be [B, q_len, heads, 128]")
    index = q.get_device()
    B, q_len, Hq, _ = q_shape
    Hkv = k_shape[2]
    q_at, q_st = _expect_rows(q, "q", q_shape, B, q_len, Hq, index)
    k_at, k_st = _expect_rows(k, "k", k_shape, B, q_len, Hkv, index)
    cache = CACHE_NONE
    v_at = v_st = kp_at = vp_at = ps = ts = hs = bt_at = bt_stride = sl_at = err = pages = 0
    if pool is not None or k_pool is not None or v_pool is not None:
        if pool is not None:
            if k_pool is not None or v_pool is not None:
                raise ValueError("either the bf16 pools or the 4-bit one")
            cache, kp, shape = CACHE_Q4, pool, pool.shape
            if pool.dtype is not _U8 or len(shape) != 4 or shape[3] != Q4_ROW_BYTES:
                raise ValueError(f"the pool must be uint8 with rows of {Q4_ROW_BYTES} bytes")
            st = pool.stride()
        else:
            if k_pool is None or v_pool is None:
                raise ValueError("k_pool and v_pool are given together")
            cache, kp, shape = CACHE_BF16, k_pool, k_pool.shape
            if k_pool.dtype is not _BF16 or len(shape) != 4 or shape[3] != 128:
                raise ValueError("k_pool must be bf16 with rows of 128 elements")
            st = k_pool.stride()
            vp_at = _expect(v_pool, "v_pool", _BF16, shape, index, False)
            if v_pool.stride() != st:
                raise ValueError("K and V pools must share strides")
        if v is None or block_table is None or seq_lens is None:
            raise ValueError("storing in a cache needs v, block_table and seq_lens")
        if kp.get_device() != index:
            raise ValueError(f"the pool is on {kp.device}, q on device {index}")
        slots, heads, ps, ts, hs = _pool_layout(shape, st, layout)
        if slots != page_size or heads != Hkv:
            raise ValueError(f"the pool holds {slots} slots per page and {heads} heads; page_size "
                             f"is {page_size}, k has {Hkv} heads")
        v_at, v_st = _expect_rows(v, "v", v.shape, B, q_len, Hkv, index)
        rows, bt_at, bt_stride, sl_at, err = _expect_table(block_table, seq_lens, index, err_flags)
        if rows != B:
            raise ValueError(f"block_table has {rows} rows for {B} sequences")
        kp_at, pages = kp.data_ptr(), shape[0]
    elif seq_lens is not None:
        sl_at = _expect(seq_lens, "seq_lens", _I32, (B,), index)
    if rope is None:
        rope = _NO_ROPE
    pos_at = axis_st = 0
    if positions is not None:
        shape = positions.shape
        if len(shape) == 2:
            if rope.n_axes > 1:
                raise ValueError(f"the rope follows {rope.n_axes} axes: positions must be "
                                 "[axes, B, q_len]")
            if (shape != (B, q_len) or positions.dtype is not _I32
                    or positions.get_device() != index or not positions.is_contiguous()):
                _refuse(positions, "positions", _I32, (B, q_len), index, True)
            pos_at = positions.data_ptr()
        else:
            n = shape[0] if len(shape) == 3 else 0
            if n < rope.n_axes:
                raise ValueError(f"positions must be [B, q_len], or [axes, B, q_len] with at least "
                                 f"{rope.n_axes} axes")
            pos_at = _expect(positions, "positions", _I32, (n, B, q_len), index)
        axis_st = B * q_len
    elif rope.n_freq and not sl_at:
        raise ValueError("a rotation needs positions, or seq_lens")
    qw = kw = 0
    if q_weight is not None:
        qw = _expect(q_weight, "q_weight", _F32, (128,), index)
    if k_weight is not None:
        kw = _expect(k_weight, "k_weight", _F32, (128,), index)
    ko_at = ko_st = 0
    if q_out is not None:
        qo_at, qo_st = _expect_rows(q_out, "q_out", q_out.shape, B, q_len, Hq, index)
    if k_out is not None:
        ko_at, ko_st = _expect_rows(k_out, "k_out", k_out.shape, B, q_len, Hkv, index)
    on, scratch = _on(index, stream)
    if q_out is None or (k_out is None and not cache):
        with scratch:
            if q_out is None:
                q_out = torch.empty((B, q_len, Hq, 128), dtype=_BF16, device=q.device)
                qo_at, qo_st = q_out.data_ptr(), Hq * 128
            if k_out is None and not cache:
                k_out = torch.empty((B, q_len, Hkv, 128), dtype=_BF16, device=q.device)
                ko_at, ko_st = k_out.data_ptr(), Hkv * 128
    status = (_raw.get("zl_qk_norm_rope") or _raw_fn("zl_qk_norm_rope", 1))(_pack(
        _NORM_ROPE, _NORM_ROPE.size, q_at, k_at, v_at, q_st, k_st, v_st, qo_at, ko_at, qo_st,
        ko_st, qw, kw, eps, rope.scale, ctypes.addressof(rope._turns), ctypes.addressof(rope._axes),
        rope.n_freq, rope.n_axes, rope.interleaved, cache, pos_at, axis_st, kp_at, vp_at, ps, ts, hs,
        bt_at, bt_stride, sl_at, B, q_len, Hq, Hkv, page_size, pages, err), on)
    if status != OK:
        _check(status, "zl_qk_norm_rope")
    return q_out, k_out
