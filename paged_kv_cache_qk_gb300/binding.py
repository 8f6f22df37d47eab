"""Python binding of the pkvqk C ABI (``include/pkvqk.h``).

Argument marshalling only: the ``pkvqk_*`` functions below have the C names
and C arguments (integers for pointers, ints, floats); the short-named
helpers (``norm_rope_append``, ``paged_decode``, ``paged_prefill``,
``lse_combine``) take torch
tensors, read their data pointers and strides and call the C entry point on
the current CUDA stream.  All computation happens in the library's kernels;
if ``libpkvqk.so`` is missing or fails to load, importing this module raises.
"""

from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkvqk.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} not found: build it with `python -m paged_kv_cache_qk_gb300.build` "
        "(there is no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)

c_i32, c_i64, c_f32, c_size, c_vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p

PKVQK_OK = 0
PKVQK_ERR_INVALID_ARG = 1
PKVQK_ERR_UNSUPPORTED = 2
PKVQK_ERR_WORKSPACE_TOO_SMALL = 3
PKVQK_ERR_POINTER_RESIDENCY = 4
PKVQK_ERR_CUDA = 5
STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "WORKSPACE_TOO_SMALL",
                4: "POINTER_RESIDENCY", 5: "CUDA"}

FLAG_BAD_SLOT = 0x1
FLAG_BAD_BLOCK_ID = 0x2
FLAG_WAIT_TIMEOUT = 0x4
FLAG_BAD_VALUE = 0x8

Q8_E4M3 = 1
Q8_INT8 = 2


class CacheLayout(ctypes.Structure):
    """Mirror of ``pkvqk_cache_layout``."""
    _fields_ = [
        ("num_blocks", c_i64),
        ("block_size", c_i32),
        ("num_kv_heads", c_i32),
        ("head_dim", c_i32),
        ("reserved", c_i32),
        ("block_stride", c_i64),
        ("slot_stride", c_i64),
        ("head_stride", c_i64),
    ]


class Q8Cache(ctypes.Structure):
    """Mirror of ``pkvqk_q8_cache``."""
    _fields_ = [
        ("k", c_vp),
        ("v", c_vp),
        ("k_scales", c_vp),
        ("v_scales", c_vp),
        ("layout", CacheLayout),
        ("format", c_i32),
        ("reserved", c_i32),
        ("scale_block_stride", c_i64),
        ("scale_group_stride", c_i64),
        ("scale_head_stride", c_i64),
    ]


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


pkvqk_last_error = _sig("pkvqk_last_error", ctypes.c_char_p, [])
pkvqk_abi_version = _sig("pkvqk_abi_version", c_i32, [])
pkvqk_norm_rope_append = _sig("pkvqk_norm_rope_append", ctypes.c_int, [
    c_vp, c_i64, c_i64,                 # q, strides
    c_vp, c_i64, c_i64,                 # k
    c_vp, c_i64, c_i64,                 # v
    c_vp, c_vp,                         # positions, slot_mapping
    c_vp, c_vp,                         # gamma_q, gamma_k
    c_f32, c_f32,                       # theta, eps
    c_i32, c_i32,                       # num_tokens, num_q_heads
    c_vp, c_vp, ctypes.POINTER(CacheLayout),
    c_vp, c_vp])                        # status_flags, stream
pkvqk_rope_table_bytes = _sig("pkvqk_rope_table_bytes", c_size, [c_i32])
pkvqk_rope_table_build = _sig("pkvqk_rope_table_build", ctypes.c_int, [c_vp, c_i32, c_f32, c_vp])
pkvqk_norm_rope_append_cached = _sig("pkvqk_norm_rope_append_cached", ctypes.c_int, [
    c_vp, c_i64, c_i64,                 # q, strides
    c_vp, c_i64, c_i64,                 # k
    c_vp, c_i64, c_i64,                 # v
    c_vp, c_vp,                         # positions, slot_mapping
    c_vp, c_vp,                         # gamma_q, gamma_k
    c_f32, c_f32,                       # theta, eps
    c_i32, c_i32,                       # num_tokens, num_q_heads
    c_vp, c_vp, ctypes.POINTER(CacheLayout),
    c_vp, c_i32,                        # rope_table, table_positions
    c_vp, c_vp])                        # status_flags, stream
pkvqk_choose_num_splits = _sig("pkvqk_choose_num_splits", c_i32,
                               [c_i32, c_i32, c_i32, c_i32, c_i64, c_i32, c_i32])
pkvqk_decode_workspace_bytes = _sig("pkvqk_decode_workspace_bytes", c_size,
                                    [c_i32, c_i32, c_i32, c_i32, c_i32])
_decode_args = [
    c_vp, c_i64, c_i64,                 # q, strides
    c_vp, c_vp, ctypes.POINTER(CacheLayout),
    c_vp, c_i32,                        # block_tables, max_blocks_per_seq
    c_vp,                               # seq_lens
    c_i32, c_i32, c_i32,                # batch, q_len, num_q_heads
    c_i32, c_i32, c_f32,                # num_splits, max_seq_len_hint, scale
]
pkvqk_paged_decode = _sig("pkvqk_paged_decode", ctypes.c_int,
                          _decode_args + [c_vp, c_vp, c_vp, c_size, c_vp, c_vp])
pkvqk_paged_decode_partials = _sig("pkvqk_paged_decode_partials", ctypes.c_int,
                                   _decode_args + [c_vp, c_size, c_vp, c_vp])
pkvqk_lse_combine = _sig("pkvqk_lse_combine", ctypes.c_int,
                         [c_vp, c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp])
pkvqk_paged_decode_static_ws = _sig("pkvqk_paged_decode_static_ws", ctypes.c_int,
                                    _decode_args + [c_vp, c_vp, c_vp, c_vp])
pkvqk_static_workspace_capacity = _sig("pkvqk_static_workspace_capacity", c_size, [])
pkvqk_choose_prefill_splits = _sig("pkvqk_choose_prefill_splits", c_i32,
                                   [c_i32, c_i32, c_i32, c_i32, c_i32, c_i32])
pkvqk_prefill_workspace_bytes = _sig("pkvqk_prefill_workspace_bytes", c_size,
                                     [c_i32, c_i32, c_i32, c_i32, c_i32])
pkvqk_paged_prefill = _sig("pkvqk_paged_prefill", ctypes.c_int,
                           _decode_args + [c_vp, c_vp, c_vp, c_size, c_vp, c_vp])
pkvqk_paged_prefill_varlen = _sig("pkvqk_paged_prefill_varlen", ctypes.c_int, [
    c_vp, c_i64, c_i64,                 # q, strides
    c_vp, c_i32, c_i64,                 # cu_seqlens_q, max_q_len, total_q
    c_vp, c_vp, ctypes.POINTER(CacheLayout),
    c_vp, c_i32, c_vp,                  # block_tables, max_blocks_per_seq, seq_lens
    c_i32, c_i32,                       # batch, num_q_heads
    c_i32, c_i32, c_f32,                # num_splits, max_seq_len_hint, scale
    c_vp, c_vp, c_vp, c_size, c_vp, c_vp])

pkvqk_norm_rope_append_q8 = _sig("pkvqk_norm_rope_append_q8", ctypes.c_int, [
    c_vp, c_i64, c_i64,                 # q, strides
    c_vp, c_i64, c_i64,                 # q_out
    c_vp, c_i64, c_i64,                 # k
    c_vp, c_i64, c_i64,                 # v
    c_vp, c_vp,                         # positions, slot_mapping
    c_vp, c_vp,                         # gamma_q, gamma_k
    c_f32, c_f32,                       # theta, eps
    c_i32, c_i32,                       # num_tokens, num_q_heads
    ctypes.POINTER(Q8Cache),
    c_vp, c_i32,                        # rope_table, table_positions
    c_vp, c_vp])                        # status_flags, stream
_decode_q8_args = [
    c_vp, c_i64, c_i64,                 # q, strides
    ctypes.POINTER(Q8Cache),
    c_vp, c_i32,                        # block_tables, max_blocks_per_seq
    c_vp,                               # seq_lens
    c_i32, c_i32, c_i32,                # batch, q_len, num_q_heads
    c_i32, c_i32, c_f32,                # num_splits, max_seq_len_hint, scale
]
pkvqk_paged_decode_q8 = _sig("pkvqk_paged_decode_q8", ctypes.c_int,
                             _decode_q8_args + [c_vp, c_vp, c_vp, c_size, c_vp, c_vp])
pkvqk_paged_prefill_q8 = _sig("pkvqk_paged_prefill_q8", ctypes.c_int,
                              _decode_q8_args + [c_vp, c_vp, c_vp, c_size, c_vp, c_vp])
pkvqk_paged_prefill_varlen_q8 = _sig("pkvqk_paged_prefill_varlen_q8", ctypes.c_int, [
    c_vp, c_i64, c_i64,                 # q, strides
    c_vp, c_i32, c_i64,                 # cu_seqlens_q, max_q_len, total_q
    ctypes.POINTER(Q8Cache),
    c_vp, c_i32, c_vp,                  # block_tables, max_blocks_per_seq, seq_lens
    c_i32, c_i32,                       # batch, num_q_heads
    c_i32, c_i32, c_f32,                # num_splits, max_seq_len_hint, scale
    c_vp, c_vp, c_vp, c_size, c_vp, c_vp])

EXPORTED = [
    "pkvqk_last_error", "pkvqk_abi_version", "pkvqk_norm_rope_append",
    "pkvqk_choose_num_splits", "pkvqk_decode_workspace_bytes", "pkvqk_paged_decode",
    "pkvqk_paged_decode_partials", "pkvqk_lse_combine", "pkvqk_paged_decode_static_ws",
    "pkvqk_static_workspace_capacity", "pkvqk_choose_prefill_splits",
    "pkvqk_prefill_workspace_bytes", "pkvqk_paged_prefill", "pkvqk_paged_prefill_varlen",
    "pkvqk_rope_table_bytes", "pkvqk_rope_table_build", "pkvqk_norm_rope_append_cached",
    "pkvqk_norm_rope_append_q8", "pkvqk_paged_decode_q8", "pkvqk_paged_prefill_q8",
    "pkvqk_paged_prefill_varlen_q8",
]


class PkvqkError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"pkvqk status {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def check(status):
    if status != PKVQK_OK:
        raise PkvqkError(status, pkvqk_last_error().decode(errors="replace"))
    return status


# ---------------------------------------------------------- torch helpers

def _torch():
    import torch
    return torch


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def cache_layout(k_cache) -> CacheLayout:
    """Layout of a [num_blocks, block_size, num_kv_heads, head_dim] (strided) cache view."""
    nb, bs, hkv, d = k_cache.shape
    s = k_cache.stride()
    if s[3] != 1:
        raise ValueError("head_dim must be the contiguous axis")
    return CacheLayout(nb, bs, hkv, d, 0, s[0], s[1], s[2])


def norm_rope_append(q, k, v, positions, slot_mapping, gamma_q, gamma_k, theta, eps,
                     k_cache, v_cache, status_flags=None, stream=None):
    """q [T, Hq, D] (in place), k/v [T, Hkv, D], caches [NB, bs, Hkv, D] views."""
    T, Hq, D = q.shape
    lay = cache_layout(k_cache)
    if tuple(v_cache.stride()) != tuple(k_cache.stride()) or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must share one layout")
    check(pkvqk_norm_rope_append(
        _ptr(q), q.stride(0), q.stride(1),
        _ptr(k), k.stride(0), k.stride(1),
        _ptr(v), v.stride(0), v.stride(1),
        _ptr(positions), _ptr(slot_mapping), _ptr(gamma_q), _ptr(gamma_k),
        float(theta), float(eps), T, Hq,
        _ptr(k_cache), _ptr(v_cache), ctypes.byref(lay),
        _ptr(status_flags), _stream(stream)))


def rope_table_bytes(max_positions):
    return int(pkvqk_rope_table_bytes(max_positions))


def rope_table_build(table, max_positions, theta, stream=None):
    """table: device tensor of at least rope_table_bytes(max_positions) bytes."""
    if max_positions > 0 and table.numel() * table.element_size() < rope_table_bytes(max_positions):
        raise ValueError("rope table too small")
    check(pkvqk_rope_table_build(_ptr(table), max_positions, float(theta), _stream(stream)))


def norm_rope_append_cached(q, k, v, positions, slot_mapping, gamma_q, gamma_k, theta, eps,
                            k_cache, v_cache, rope_table, table_positions, status_flags=None,
                            stream=None):
    """norm_rope_append with the angles of positions < table_positions read from a
    table built by rope_table_build (same theta)."""
    T, Hq, D = q.shape
    lay = cache_layout(k_cache)
    if tuple(v_cache.stride()) != tuple(k_cache.stride()) or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must share one layout")
    check(pkvqk_norm_rope_append_cached(
        _ptr(q), q.stride(0), q.stride(1),
        _ptr(k), k.stride(0), k.stride(1),
        _ptr(v), v.stride(0), v.stride(1),
        _ptr(positions), _ptr(slot_mapping), _ptr(gamma_q), _ptr(gamma_k),
        float(theta), float(eps), T, Hq,
        _ptr(k_cache), _ptr(v_cache), ctypes.byref(lay),
        _ptr(rope_table), int(table_positions),
        _ptr(status_flags), _stream(stream)))


def decode_workspace_bytes(batch, q_len, num_q_heads, head_dim, num_splits):
    return int(pkvqk_decode_workspace_bytes(batch, q_len, num_q_heads, head_dim, num_splits))


def choose_num_splits(batch, num_kv_heads, rows_per_kv_head, max_seq_len, total_tokens,
                      block_size, sm_count=0):
    return int(pkvqk_choose_num_splits(batch, num_kv_heads, rows_per_kv_head, max_seq_len,
                                       total_tokens, block_size, sm_count))


def paged_decode(q, k_cache, v_cache, block_tables, seq_lens, out, *, q_len=1, num_splits=1,
                 max_seq_len_hint=0, scale=0.0, lse_out=None, workspace=None,
                 status_flags=None, stream=None):
    """q [B*q_len, Hq, D]; out [B, q_len, Hq, D] (or [B*q_len, Hq, D]) contiguous bf16."""
    Tq, Hq, D = q.shape
    B = Tq // q_len
    lay = cache_layout(k_cache)
    if tuple(v_cache.stride()) != tuple(k_cache.stride()) or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must share one layout")
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(pkvqk_paged_decode(
        _ptr(q), q.stride(0), q.stride(1),
        _ptr(k_cache), _ptr(v_cache), ctypes.byref(lay),
        _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens),
        B, q_len, Hq, int(num_splits), int(max_seq_len_hint), float(scale),
        _ptr(out), _ptr(lse_out), _ptr(workspace), ws_bytes,
        _ptr(status_flags), _stream(stream)))


def paged_decode_partials(q, k_cache, v_cache, block_tables, seq_lens, workspace, *, q_len=1,
                          num_splits=2, max_seq_len_hint=0, scale=0.0, status_flags=None,
                          stream=None):
    Tq, Hq, D = q.shape
    B = Tq // q_len
    lay = cache_layout(k_cache)
    ws_bytes = workspace.numel() * workspace.element_size()
    check(pkvqk_paged_decode_partials(
        _ptr(q), q.stride(0), q.stride(1),
        _ptr(k_cache), _ptr(v_cache), ctypes.byref(lay),
        _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens),
        B, q_len, Hq, int(num_splits), int(max_seq_len_hint), float(scale),
        _ptr(workspace), ws_bytes, _ptr(status_flags), _stream(stream)))


def lse_combine(ws_o, ws_lse, rows, num_splits, out, lse_out=None, stream=None):
    check(pkvqk_lse_combine(_ptr(ws_o), _ptr(ws_lse), int(rows), 128, int(num_splits),
                            _ptr(out), _ptr(lse_out), _stream(stream)))


def choose_prefill_splits(batch, num_kv_heads, q_len, group, max_seq_len, sm_count=0):
    return int(pkvqk_choose_prefill_splits(batch, num_kv_heads, q_len, group, max_seq_len,
                                           sm_count))


def prefill_workspace_bytes(batch, q_len, num_q_heads, head_dim, num_splits):
    return int(pkvqk_prefill_workspace_bytes(batch, q_len, num_q_heads, head_dim, num_splits))


def paged_prefill(q, k_cache, v_cache, block_tables, seq_lens, out, *, q_len, num_splits=1,
                  max_seq_len_hint=0, scale=0.0, lse_out=None, workspace=None,
                  status_flags=None, stream=None):
    """Causal multi-query attention on the tensor cores.

    q [B*q_len, Hq, D]; out [B, q_len, Hq, D] (or [B*q_len, Hq, D]) contiguous bf16.
    """
    Tq, Hq, D = q.shape
    B = Tq // q_len
    lay = cache_layout(k_cache)
    if tuple(v_cache.stride()) != tuple(k_cache.stride()) or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must share one layout")
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(pkvqk_paged_prefill(
        _ptr(q), q.stride(0), q.stride(1),
        _ptr(k_cache), _ptr(v_cache), ctypes.byref(lay),
        _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens),
        B, q_len, Hq, int(num_splits), int(max_seq_len_hint), float(scale),
        _ptr(out), _ptr(lse_out), _ptr(workspace), ws_bytes,
        _ptr(status_flags), _stream(stream)))


def paged_prefill_varlen(q, cu_seqlens_q, max_q_len, k_cache, v_cache, block_tables, seq_lens,
                         out, *, num_splits=1, max_seq_len_hint=0, scale=0.0, lse_out=None,
                         workspace=None, status_flags=None, stream=None):
    """Varlen causal multi-query attention on the tensor cores.

    q [total_q, Hq, D] packed rows, cu_seqlens_q int32 [B + 1] on the device,
    max_q_len a host int; out [total_q, Hq, D] contiguous bf16.
    """
    total_q, Hq, D = q.shape
    B = cu_seqlens_q.shape[0] - 1
    lay = cache_layout(k_cache)
    if tuple(v_cache.stride()) != tuple(k_cache.stride()) or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must share one layout")
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(pkvqk_paged_prefill_varlen(
        _ptr(q), q.stride(0), q.stride(1), _ptr(cu_seqlens_q), int(max_q_len), int(total_q),
        _ptr(k_cache), _ptr(v_cache), ctypes.byref(lay),
        _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens),
        B, Hq, int(num_splits), int(max_seq_len_hint), float(scale),
        _ptr(out), _ptr(lse_out), _ptr(workspace), ws_bytes,
        _ptr(status_flags), _stream(stream)))


# ------------------------------------------------------------- 8-bit caches
#
# These calls are a few microseconds of kernel at decode sizes, so the host side
# is kept short: the cache's description is packed in one go, strides are read
# once a tensor, and the current stream is asked for by its handle.

_Q8_PACK = struct.Struct("=4Qq4i3q2i3q")       # pkvqk_q8_cache, no padding
assert _Q8_PACK.size == ctypes.sizeof(Q8Cache)
_q8 = {}                                       # torch names, filled on first use
_ROPE_ROW_BYTES = pkvqk_rope_table_bytes(1)


def _q8_names():
    torch = _torch()
    _q8.update(formats={torch.float8_e4m3fn: Q8_E4M3, torch.int8: Q8_INT8},
               bf16=torch.bfloat16, f32=torch.float32, i32=torch.int32, i64=torch.int64,
               raw_stream=torch._C._cuda_getCurrentRawStream)
    return _q8


def _fast(name, args):
    """The entry point with the cache passed as packed bytes."""
    f = _lib[name]
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.c_char_p if a is ctypes.POINTER(Q8Cache) else a for a in args]
    return f


_append_q8 = _fast("pkvqk_norm_rope_append_q8", pkvqk_norm_rope_append_q8.argtypes)
_paged_decode_q8 = _fast("pkvqk_paged_decode_q8", pkvqk_paged_decode_q8.argtypes)
_paged_prefill_q8 = _fast("pkvqk_paged_prefill_q8", pkvqk_paged_prefill_q8.argtypes)
_paged_prefill_varlen_q8 = _fast("pkvqk_paged_prefill_varlen_q8",
                                 pkvqk_paged_prefill_varlen_q8.argtypes)


def _pack_q8(t, k_cache, v_cache, k_scales, v_scales):
    shape, st = k_cache.shape, k_cache.stride()
    fmt = t["formats"].get(k_cache.dtype)
    if fmt is None or v_cache.dtype is not k_cache.dtype:
        raise ValueError("k_cache and v_cache must both be float8_e4m3fn or int8")
    if v_cache.stride() != st or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must share one layout")
    nb, bs, hkv, d = shape
    if st[3] != 1:
        raise ValueError("head_dim must be the contiguous axis")
    if k_scales.dtype is not t["f32"] or v_scales.dtype is not t["f32"]:
        raise ValueError("scales must be float32")
    ss = k_scales.stride()
    if k_scales.shape != (nb, bs // 16, hkv) or v_scales.shape != k_scales.shape \
            or v_scales.stride() != ss:
        raise ValueError("scales must be [num_blocks, block_size // 16, num_kv_heads] "
                         "and share one layout")
    # an axis of length 1 is never stepped along: any positive stride will do
    return _Q8_PACK.pack(
        k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
        nb, bs, hkv, d, 0, st[0], st[1], st[2], fmt, 0,
        ss[0] if nb > 1 else ss[0] or 1, ss[1] if bs > 16 else ss[1] or 1,
        ss[2] if hkv > 1 else ss[2] or 1)


def q8_cache(k_cache, v_cache, k_scales, v_scales) -> Q8Cache:
    """The C description of an 8-bit cache.

    k_cache, v_cache: [num_blocks, block_size, num_kv_heads, head_dim] views of one
    layout, float8_e4m3fn or int8; k_scales, v_scales: fp32 [num_blocks,
    block_size // 16, num_kv_heads] views of one layout.
    """
    return Q8Cache.from_buffer_copy(_pack_q8(_q8 or _q8_names(), k_cache, v_cache, k_scales,
                                             v_scales))


def _heads(t, x, name):
    """(tokens, heads, token stride, head stride) of a [tokens, heads, head_dim] view."""
    n, h, d = x.shape
    s0, s1, s2 = x.stride()
    if x.dtype is not t["bf16"] or d != 128 or s2 != 1:
        raise ValueError(f"{name} must be bfloat16 with a head_dim of 128, the contiguous axis")
    return n, h, s0, s1


def _gains(t, x, name):
    if x.dtype is not t["bf16"] or x.numel() != 128 or not x.is_contiguous():
        raise ValueError(f"{name} must be 128 contiguous bfloat16 values")
    return x.data_ptr()


def _ints(x, dtype, n, name):
    if x.dtype is not dtype or not x.is_contiguous() or x.numel() != n:
        raise ValueError(f"{name} must be {n} contiguous {dtype} values")
    return x.data_ptr()


def _results(t, out, lse_out, rows, heads):
    """Pointers of out [rows, heads, head_dim] and lse_out [rows, heads] (or None); both
    may hold more rows, which are left as they are."""
    if out.dtype is not t["bf16"] or not out.is_contiguous() or out.numel() < rows * heads * 128:
        raise ValueError("out must be contiguous bfloat16, one value per value of q")
    if lse_out is None:
        return out.data_ptr(), 0
    if lse_out.dtype is not t["f32"] or not lse_out.is_contiguous() \
            or lse_out.numel() < rows * heads:
        raise ValueError("lse_out must be contiguous float32, one value per row and head")
    return out.data_ptr(), lse_out.data_ptr()


def _flags(t, x):
    if x is None:
        return 0
    if x.dtype is not t["i32"] or x.numel() < 1:
        raise ValueError("status_flags must be int32")
    return x.data_ptr()


def _workspace(x):
    """Pointer and bytes of a workspace (or None)."""
    if x is None:
        return 0, 0
    if not x.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return x.data_ptr(), x.nbytes


def _table(t, block_tables, batch):
    if block_tables.dtype is not t["i32"] or block_tables.shape[0] != batch \
            or not block_tables.is_contiguous():
        raise ValueError("block_tables must be contiguous int32 [batch, max_blocks_per_seq]")
    return block_tables.data_ptr(), block_tables.shape[1]


def _raw_stream(t, stream, x):
    if stream is not None:
        return stream.cuda_stream
    index = x.get_device()
    return t["raw_stream"](index) if index >= 0 else 0   # a host tensor is refused below


def norm_rope_append_q8(q, k, v, positions, slot_mapping, gamma_q, gamma_k, theta, eps,
                        k_cache, v_cache, k_scales, v_scales, *, q_out=None, rope_table=None,
                        table_positions=0, status_flags=None, stream=None):
    """norm_rope_append into an 8-bit cache (see q8_cache); q [T, Hq, D] is written to
    q_out (default: in place).  rope_table as for norm_rope_append_cached."""
    t = _q8 or _q8_names()
    q_out = q if q_out is None else q_out
    T, Hq, qs, qh = _heads(t, q, "q")
    To, Ho, os_, oh = _heads(t, q_out, "q_out")
    Tk, Hk, ks, kh = _heads(t, k, "k")
    Tv, Hv, vs, vh = _heads(t, v, "v")
    if (To, Ho) != (T, Hq) or Tk != T or Tv != T or Hk != Hv or Hk != k_cache.shape[2]:
        raise ValueError("q, q_out, k and v must agree in tokens, and k, v and the cache in heads")
    if rope_table is not None and (not rope_table.is_contiguous()
                                   or rope_table.nbytes < table_positions * _ROPE_ROW_BYTES):
        raise ValueError(f"rope_table must be contiguous and hold {table_positions} positions")
    check(_append_q8(
        q.data_ptr(), qs, qh, q_out.data_ptr(), os_, oh, k.data_ptr(), ks, kh,
        v.data_ptr(), vs, vh, _ints(positions, t["i64"], T, "positions"),
        _ints(slot_mapping, t["i64"], T, "slot_mapping"), _gains(t, gamma_q, "gamma_q"),
        _gains(t, gamma_k, "gamma_k"), theta, eps, T, Hq,
        _pack_q8(t, k_cache, v_cache, k_scales, v_scales), _ptr(rope_table), table_positions,
        _flags(t, status_flags), _raw_stream(t, stream, q)))


def _attend_q8(f, q, caches, block_tables, seq_lens, out, q_len, num_splits, max_seq_len_hint,
               scale, lse_out, workspace, status_flags, stream):
    t = _q8 or _q8_names()
    rows, Hq, qs, qh = _heads(t, q, "q")
    batch = seq_lens.shape[0]
    if q_len * batch != rows:
        raise ValueError("q must hold q_len rows for each sequence of seq_lens")
    table, width = _table(t, block_tables, batch)
    o, lse = _results(t, out, lse_out, rows, Hq)
    check(f(
        q.data_ptr(), qs, qh, _pack_q8(t, *caches), table, width,
        _ints(seq_lens, t["i32"], batch, "seq_lens"), batch, q_len, Hq, num_splits,
        max_seq_len_hint, scale, o, lse, *_workspace(workspace), _flags(t, status_flags),
        _raw_stream(t, stream, q)))


def paged_decode_q8(q, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens, out, *,
                    q_len=1, num_splits=1, max_seq_len_hint=0, scale=0.0, lse_out=None,
                    workspace=None, status_flags=None, stream=None):
    """paged_decode over an 8-bit cache (see q8_cache)."""
    _attend_q8(_paged_decode_q8, q, (k_cache, v_cache, k_scales, v_scales), block_tables,
               seq_lens, out, q_len, num_splits, max_seq_len_hint, scale, lse_out, workspace,
               status_flags, stream)


def paged_prefill_q8(q, k_cache, v_cache, k_scales, v_scales, block_tables, seq_lens, out, *,
                     q_len, num_splits=1, max_seq_len_hint=0, scale=0.0, lse_out=None,
                     workspace=None, status_flags=None, stream=None):
    """paged_prefill over an 8-bit cache (see q8_cache)."""
    _attend_q8(_paged_prefill_q8, q, (k_cache, v_cache, k_scales, v_scales), block_tables,
               seq_lens, out, q_len, num_splits, max_seq_len_hint, scale, lse_out, workspace,
               status_flags, stream)


def paged_prefill_varlen_q8(q, cu_seqlens_q, max_q_len, k_cache, v_cache, k_scales, v_scales,
                            block_tables, seq_lens, out, *, num_splits=1, max_seq_len_hint=0,
                            scale=0.0, lse_out=None, workspace=None, status_flags=None,
                            stream=None):
    """paged_prefill_varlen over an 8-bit cache (see q8_cache)."""
    t = _q8 or _q8_names()
    total_q, Hq, qs, qh = _heads(t, q, "q")
    batch = seq_lens.shape[0]
    table, width = _table(t, block_tables, batch)
    o, lse = _results(t, out, lse_out, total_q, Hq)
    check(_paged_prefill_varlen_q8(
        q.data_ptr(), qs, qh, _ints(cu_seqlens_q, t["i32"], batch + 1, "cu_seqlens_q"), max_q_len,
        total_q, _pack_q8(t, k_cache, v_cache, k_scales, v_scales), table, width,
        _ints(seq_lens, t["i32"], batch, "seq_lens"), batch, Hq, num_splits, max_seq_len_hint,
        scale, o, lse, *_workspace(workspace), _flags(t, status_flags),
        _raw_stream(t, stream, q)))
