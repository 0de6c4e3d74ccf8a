"""Python binding of ``libpa.so`` (include/paged_attention.h).

Argument marshalling only: tensors are turned into device pointers and sizes
and handed to the C ABI on the current CUDA stream.  Every step of the path
runs in the library's CUDA kernels; there is no fallback.  If the library has
not been built, :func:`library` raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

# PA_LIBRARY selects another build of the library (e.g. a tuning variant)
_LIB_PATH = os.environ.get("PA_LIBRARY") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libpa.so")

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_ERR_CUDA = range(5)
PA_F32, PA_BF16 = 0, 1

ERRBIT_BLOCK_ID = 1
ERRBIT_CONTEXT_LEN = 2
ERRBIT_SLOT = 4
ERRBIT_PAIR = 8
ERRBIT_TIMEOUT = 16
ERRBIT_QUERY = 32
ERRBIT_GROUP = 64
ERRBIT_AXIS = 128

EXPORTED = ("pa_status_str", "pa_decode_workspace_size", "pa_decode_workspace_init",
            "pa_decode_launch_config", "pa_decode", "pa_decode_noalloc", "pa_decode_append",
            "pa_prefill", "pa_prefill_workspace_size", "pa_prefill_launch_config",
            "pa_reshape_and_cache", "pa_copy_blocks", "pa_shared_prefix_plan",
            "pa_shared_prefix_plan_tree",
            "pa_shared_prefix_workspace_size", "pa_decode_shared_prefix", "pa_rope_append",
            "pa_rope_append_packed", "pa_cross_attention", "pa_cross_attention_packed",
            "pa_cross_attention_workspace_size")

# size of the library's fixed scratch array used by pa_decode_noalloc
NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


class PagedAttentionError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_str(status)}")
        self.status = status


_lib: Optional[ctypes.CDLL] = None


def library(path: Optional[str] = None) -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with `python -m paged_kv_cache_456_b200.build`"
                           " (the CUDA library is the only implementation)")
    lib = ctypes.CDLL(p)
    vp, i, sz, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    lib.pa_status_str.argtypes = [i]
    lib.pa_status_str.restype = ctypes.c_char_p
    lib.pa_decode_workspace_size.argtypes = [i] * 7 + [ctypes.POINTER(sz)]
    lib.pa_decode_workspace_size.restype = i
    lib.pa_decode_workspace_init.argtypes = [vp, sz, vp]
    lib.pa_decode_workspace_init.restype = i
    lib.pa_decode_launch_config.argtypes = [i] * 7 + [ctypes.POINTER(i)] * 4
    lib.pa_decode_launch_config.restype = i
    lib.pa_decode.argtypes = [vp] * 6 + [i] * 8 + [f, i, i, vp, sz, vp, vp]
    lib.pa_decode.restype = i
    lib.pa_decode_noalloc.argtypes = [vp] * 6 + [i] * 8 + [f, i, i, vp, vp]
    lib.pa_prefill_launch_config.restype = i
    lib.pa_prefill_launch_config.argtypes = [i] * 8 + [ctypes.POINTER(i)] * 4
    lib.pa_prefill_workspace_size.restype = i
    lib.pa_prefill_workspace_size.argtypes = [i] * 8 + [ctypes.POINTER(sz)]
    lib.pa_prefill.restype = i
    lib.pa_prefill.argtypes = [vp] * 7 + [i] * 9 + [f, i, i, vp, sz, vp, vp]
    lib.pa_decode_append.restype = i
    lib.pa_decode_append.argtypes = [vp] * 8 + [i] * 8 + [f, i, i, vp, sz, vp, vp]
    lib.pa_decode_noalloc.restype = i
    lib.pa_reshape_and_cache.argtypes = [vp] * 5 + [i] * 6 + [vp, vp]
    lib.pa_reshape_and_cache.restype = i
    lib.pa_copy_blocks.argtypes = [vp] * 3 + [i] * 6 + [vp, vp]
    lib.pa_copy_blocks.restype = i
    i64 = ctypes.c_int64
    lib.pa_rope_append.argtypes = [vp] * 10 + [i] * 3 + [f] + [i64] * 4 + [i] * 7 + [vp, vp]
    lib.pa_rope_append.restype = i
    lib.pa_cross_attention_workspace_size.argtypes = [i] * 7 + [ctypes.POINTER(sz)]
    lib.pa_cross_attention_workspace_size.restype = i
    lib.pa_cross_attention.argtypes = [vp] * 7 + [i] * 9 + [f, i, vp, sz, vp, vp]
    lib.pa_cross_attention.restype = i
    for fn in (lib.pa_rope_append_packed, lib.pa_cross_attention_packed):
        fn.argtypes = [ctypes.c_char_p]
        fn.restype = i
    ip = ctypes.POINTER(i)
    lib.pa_shared_prefix_plan.argtypes = [vp, vp] + [i] * 4 + [vp, vp, vp, ip, ip]
    lib.pa_shared_prefix_plan.restype = i
    lib.pa_shared_prefix_plan_tree.argtypes = [vp, vp] + [i] * 4 + [vp, vp, vp, ip, ip]
    lib.pa_shared_prefix_plan_tree.restype = i
    lib.pa_shared_prefix_workspace_size.argtypes = [i] * 9 + [ctypes.POINTER(sz)]
    lib.pa_shared_prefix_workspace_size.restype = i
    lib.pa_decode_shared_prefix.argtypes = [vp] * 11 + [i] * 10 + [f, i, i, vp, sz, vp, vp]
    lib.pa_decode_shared_prefix.restype = i
    if path is None:
        _lib = lib
    return lib


def status_str(status: int) -> str:
    return library().pa_status_str(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != PA_OK:
        raise PagedAttentionError(status, what)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return PA_BF16
    if t.dtype == torch.float32:
        return PA_F32
    raise TypeError(f"unsupported element type {t.dtype} (float32 or bfloat16)")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libpa must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _call_on(dev: int, fn, what: str, stream, layout, *args) -> None:
    """``fn`` of ``args`` and the stream (the current one by default) packed into its argument
    struct, with device ``dev`` current.  (One pointer for ctypes to convert in the place of 22 to
    27 values: rope_append of one token takes 10.8 us in the place of 13.0.)"""
    if stream is None:
        stream = _raw_stream(dev)
    else:
        stream = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    try:
        packed = layout.pack(*args, stream)
    except struct.error as e:
        raise ValueError(f"{what}: an argument is out of its type's range: {e}") from None
    if torch.cuda.current_device() == dev:
        status = fn(packed)
    else:
        with torch.cuda.device(dev):
            status = fn(packed)
    if status != PA_OK:
        raise PagedAttentionError(status, what)


def _raw_stream(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


# the fields of pa_rope_append_args and pa_cross_attention_args, aligned as C does
_ROPE_ARGS = struct.Struct("10P4qP3if7iP")
_CROSS_ARGS = struct.Struct("8PNP9ifiP")

# (the handle without a Stream object around it, where this torch has it)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


# The entry points that take apart what they are given check every tensor that they hand on (a host
# pointer would fault in the kernel).  At a few microseconds of device time a call, the checks are
# kept cheap: device indexes rather than device objects, one look at a tensor.
def _device(ref: torch.Tensor) -> int:
    dev = ref.get_device()
    if dev < 0:
        raise ValueError("libpa works on CUDA tensors")
    return dev


def _refuse(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, dev: int, layout: str):
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    raise ValueError(f"{name} must be {layout} {dtype} of shape {tuple(shape)}, "
                     f"not {t.dtype} of shape {tuple(t.shape)} and strides {t.stride()}")


def _rows_ptr(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, dev: int = -1):
    """(pointer, elements between tokens) of ``[T][H][D]`` rows whose heads lie side by side."""
    T, H, D = shape
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(name, t, shape, dtype, dev, "(in each token) contiguous")
    token, head, dim = t.stride()
    if (dim != 1 and D > 1) or (head != D and H > 1):
        _refuse(name, t, shape, dtype, dev, "(in each token) contiguous")
    return t.data_ptr(), token if T > 1 else H * D


def _array_ptr(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, dev: int = -1) -> int:
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _refuse(name, t, shape, dtype, dev, "contiguous")
    return t.data_ptr()


def _err_ptr(dev: int, t: Optional[torch.Tensor]) -> int:
    if t is None:
        return 0
    if t.get_device() != dev or t.dtype is not torch.int32 or t.numel() < 1:
        raise ValueError("err_flag must be an int32 word on the device of the other tensors")
    return t.data_ptr()


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
def workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                   max_context_len: int, partition_size: int = 0,
                   dtype: torch.dtype = torch.bfloat16) -> int:
    out = ctypes.c_size_t(0)
    code = PA_BF16 if dtype == torch.bfloat16 else PA_F32
    _check(library().pa_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                              max_context_len, partition_size, code,
                                              ctypes.byref(out)), "pa_decode_workspace_size")
    return int(out.value)


def make_workspace(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                   max_context_len: int, partition_size: int = 0,
                   dtype: torch.dtype = torch.bfloat16, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of the size ``pa_decode`` needs."""
    n = workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                       partition_size, dtype)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def make_prefill_workspace(num_seqs: int, num_query_tokens: int, num_q_heads: int,
                           num_kv_heads: int, head_dim: int, max_context_len: int,
                           partition_size: int = 0, dtype: torch.dtype = torch.bfloat16,
                           device="cuda") -> torch.Tensor:
    """A zero-filled workspace of the size ``pa_prefill`` needs."""
    n = ctypes.c_size_t(0)
    _check(library().pa_prefill_workspace_size(
        num_seqs, num_query_tokens, num_q_heads, num_kv_heads, head_dim, int(max_context_len),
        int(partition_size), PA_BF16 if dtype == torch.bfloat16 else PA_F32, ctypes.byref(n)),
        "pa_prefill_workspace_size")
    return torch.zeros(max(n.value, 16), dtype=torch.uint8, device=device)


def launch_config(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                  max_context_len: int, partition_size: int = 0,
                  dtype: torch.dtype = torch.bfloat16) -> dict:
    vals = [ctypes.c_int(0) for _ in range(4)]
    code = PA_BF16 if dtype == torch.bfloat16 else PA_F32
    _check(library().pa_decode_launch_config(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                             max_context_len, partition_size, code,
                                             *[ctypes.byref(v) for v in vals]),
           "pa_decode_launch_config")
    return dict(zip(("grid", "warps_per_cta", "pipeline_depth", "smem_bytes"),
                    (v.value for v in vals)))


def prefill_launch_config(num_seqs: int, num_query_tokens: int, num_q_heads: int,
                          num_kv_heads: int, head_dim: int, max_context_len: int,
                          partition_size: int = 0, dtype: torch.dtype = torch.bfloat16) -> dict:
    vals = [ctypes.c_int(0) for _ in range(4)]
    code = PA_BF16 if dtype == torch.bfloat16 else PA_F32
    _check(library().pa_prefill_launch_config(num_seqs, num_query_tokens, num_q_heads,
                                              num_kv_heads, head_dim, max_context_len,
                                              partition_size, code,
                                              *[ctypes.byref(v) for v in vals]),
           "pa_prefill_launch_config")
    return dict(zip(("grid", "warps_per_cta", "pipeline_depth", "smem_bytes"),
                    (v.value for v in vals)))


def decode(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           block_tables: torch.Tensor, context_lens: torch.Tensor, *, scale: float,
           max_context_len: int, workspace: torch.Tensor, partition_size: int = 0,
           err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """PagedAttention decode into ``out`` ``[S][Hq][D]``; see ``pa_decode``."""
    S, Hq, D = q.shape
    N, Hkv, bs, _ = k_cache.shape
    _check(library().pa_decode(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        S, Hq, Hkv, D, bs, block_tables.shape[1], N, int(max_context_len), float(scale),
        int(partition_size), _dtype_code(q), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(err_flag), _stream(stream)), "pa_decode")
    return out


def decode_append(out: torch.Tensor, q: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                  k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                  context_lens: torch.Tensor, *, scale: float, max_context_len: int,
                  workspace: torch.Tensor, partition_size: int = 0,
                  err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Write each sequence's newest ``key``/``value`` row ``[S][Hkv][D]`` into its
    cache slot and decode over it in the same launch; see ``pa_decode_append``."""
    S, Hq, D = q.shape
    N, Hkv, bs, _ = k_cache.shape
    _check(library().pa_decode_append(
        _ptr(out), _ptr(q), _ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_tables), _ptr(context_lens), S, Hq, Hkv, D, bs, block_tables.shape[1], N,
        int(max_context_len), float(scale), int(partition_size), _dtype_code(q), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(err_flag), _stream(stream)),
        "pa_decode_append")
    return out


def prefill(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
            block_tables: torch.Tensor, context_lens: torch.Tensor, query_start: torch.Tensor, *,
            scale: float, max_context_len: int, workspace: torch.Tensor, partition_size: int = 0,
            err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention of ``q`` ``[T][Hq][D]``, the last ``query_start[s+1] -
    query_start[s]`` tokens of each sequence, into ``out``; see ``pa_prefill``.
    The workspace is sized for ``T`` query rows (``make_workspace(T, ...)``)."""
    T, Hq, D = q.shape
    N, Hkv, bs, _ = k_cache.shape
    _check(library().pa_prefill(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        _ptr(query_start), block_tables.shape[0], T, Hq, Hkv, D, bs, block_tables.shape[1], N,
        int(max_context_len), float(scale), int(partition_size), _dtype_code(q),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(err_flag),
        _stream(stream)), "pa_prefill")
    return out


def make_cross_attention_workspace(num_seqs: int, num_query_tokens: int, num_q_heads: int,
                                   num_kv_heads: int, head_dim: int, max_context_len: int,
                                   dtype: torch.dtype = torch.bfloat16, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for ``pa_cross_attention`` calls of at most ``num_query_tokens`` rows, of
    any number of sequences."""
    n = ctypes.c_size_t(0)
    with torch.cuda.device(device):
        _check(library().pa_cross_attention_workspace_size(
            num_seqs, num_query_tokens, num_q_heads, num_kv_heads, head_dim, int(max_context_len),
            PA_BF16 if dtype == torch.bfloat16 else PA_F32, ctypes.byref(n)),
            "pa_cross_attention_workspace_size")
    return torch.zeros(max(n.value, 16), dtype=torch.uint8, device=device)


def cross_attention(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                    v_cache: torch.Tensor, block_tables: torch.Tensor,
                    context_lens: torch.Tensor, query_start: torch.Tensor, *, scale: float,
                    max_context_len: int, workspace: torch.Tensor,
                    err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of each sequence's rows of ``q`` ``[T][Hq][D]`` (rows ``query_start[s]`` to
    ``query_start[s+1]``) to all ``context_lens[s]`` tokens of its block table, into ``out``;
    see ``pa_cross_attention``."""
    dev, dt, i32 = _device(q), q.dtype, torch.int32
    shape, cache, table = q.shape, k_cache.shape, block_tables.shape
    if len(shape) != 3 or len(cache) != 4 or len(table) != 2:
        raise ValueError("q is [rows][heads][head_dim], the caches [blocks][heads][16][head_dim], "
                         "block_tables [sequences][blocks]")
    T, Hq, D = shape
    N, Hkv, bs, _ = cache
    S, B = table
    cache = (N, Hkv, bs, D)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the device of the other tensors")
    _call_on(dev, library().pa_cross_attention_packed, "pa_cross_attention", stream, _CROSS_ARGS,
             _array_ptr("out", out, shape, dt, dev), _array_ptr("q", q, shape, dt, dev),
             _array_ptr("k_cache", k_cache, cache, dt, dev),
             _array_ptr("v_cache", v_cache, cache, dt, dev),
             _array_ptr("block_tables", block_tables, table, i32, dev),
             _array_ptr("context_lens", context_lens, (S,), i32, dev),
             _array_ptr("query_start", query_start, (S + 1,), i32, dev), workspace.data_ptr(),
             workspace.nbytes, _err_ptr(dev, err_flag), S, T, Hq, Hkv, D, bs, B, N,
             int(max_context_len), scale, _dtype_code(q))
    return out


def decode_noalloc(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                   *, scale: float, max_context_len: int, partition_size: int = 0,
                   err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``decode`` for callers that cannot allocate device memory: the scratch
    comes from the library's fixed array (``NOALLOC_SCRATCH_BYTES``), shared by
    every call; see ``pa_decode_noalloc``."""
    S, Hq, D = q.shape
    N, Hkv, bs, _ = k_cache.shape
    _check(library().pa_decode_noalloc(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        S, Hq, Hkv, D, bs, block_tables.shape[1], N, int(max_context_len), float(scale),
        int(partition_size), _dtype_code(q), _ptr(err_flag), _stream(stream)), "pa_decode_noalloc")
    return out


# ---------------------------------------------------------------------------
# cache maintenance
# ---------------------------------------------------------------------------
def reshape_and_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                      err_flag: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write ``key``/``value`` ``[T][Hkv][D]`` into the cache slots of ``slot_mapping``."""
    T = key.shape[0]
    N, Hkv, bs, D = k_cache.shape
    _check(library().pa_reshape_and_cache(
        _ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache), _ptr(slot_mapping), T, Hkv, D, bs, N,
        _dtype_code(k_cache), _ptr(err_flag), _stream(stream)), "pa_reshape_and_cache")


def rope_append(q_out: Optional[torch.Tensor], q: Optional[torch.Tensor],
                key: Optional[torch.Tensor], value: Optional[torch.Tensor],
                k_cache: Optional[torch.Tensor], v_cache: Optional[torch.Tensor],
                slot_mapping: Optional[torch.Tensor], positions: torch.Tensor,
                inv_freq: torch.Tensor, *, pair_axis: Optional[torch.Tensor] = None,
                adjacent: bool = False, rot_scale: float = 1.0,
                err_flag: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Turn ``q`` ``[T][Hq][D]`` by the tokens' positions into ``q_out`` and write the
    turned ``key`` and the ``value`` ``[T][Hkv][D]`` into their cache slots; see
    ``pa_rope_append``.  ``positions`` is int64 ``[T]`` or ``[axes][T]``; ``2 *
    len(inv_freq)`` dims of a head are turned, in pairs of its two halves, or of
    neighbours with ``adjacent``.  ``q``/``q_out`` may be one tensor, or both None;
    ``key`` to ``slot_mapping`` may all be None.  q, q_out, key and value may be
    views whose tokens lie apart."""
    ref = q if q is not None else key
    if ref is None:
        raise ValueError("rope_append needs q or key")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if ((value is None) != (key is None) or (k_cache is None) != (key is None)
            or (v_cache is None) != (key is None) or (slot_mapping is None) != (key is None)):
        raise ValueError("key, value, k_cache, v_cache and slot_mapping go together")
    shape, pos_shape, half = ref.shape, positions.shape, inv_freq.numel()
    if len(shape) != 3:
        raise ValueError("q and key are [tokens][heads][head_dim]")
    dev, dt, i64 = _device(ref), ref.dtype, torch.int64
    T, _, D = shape
    axes = 1 if len(pos_shape) == 1 else pos_shape[0]
    pos = _array_ptr("positions", positions, (T,) if len(pos_shape) == 1 else (axes, T), i64, dev)
    freq = _array_ptr("inv_freq", inv_freq, (half,), torch.float32, dev)
    axis = 0 if pair_axis is None else _array_ptr("pair_axis", pair_axis, (half,), torch.int32, dev)
    qp = qs = op = os_ = kp = ks = vp = vs = kc = vc = slots = Hq = Hkv = N = 0
    bs = 1
    if q is not None:
        Hq = shape[1]
        qp, qs = _rows_ptr("q", q, shape, dt, dev)
        op, os_ = _rows_ptr("q_out", q_out, shape, dt, dev)
    if key is not None:
        N, Hkv, bs, _ = k_cache.shape
        rows, cache = (T, Hkv, D), (N, Hkv, bs, D)
        kp, ks = _rows_ptr("key", key, rows, dt, dev)
        vp, vs = _rows_ptr("value", value, rows, dt, dev)
        kc = _array_ptr("k_cache", k_cache, cache, dt, dev)
        vc = _array_ptr("v_cache", v_cache, cache, dt, dev)
        slots = _array_ptr("slot_mapping", slot_mapping, (T,), i64, dev)
    _call_on(dev, library().pa_rope_append_packed, "pa_rope_append", stream, _ROPE_ARGS, op, qp, kp,
             vp, kc, vc, slots, pos, freq, axis, os_, qs, ks, vs, _err_ptr(dev, err_flag), axes,
             2 * half, adjacent, rot_scale, T, Hq, Hkv, D, bs, N, _dtype_code(ref))
    return q_out


def copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, block_mapping: torch.Tensor,
                err_flag: Optional[torch.Tensor] = None, stream=None) -> None:
    """Copy whole blocks ``src -> dst`` for each row of ``block_mapping`` ``[M][2]``."""
    N, Hkv, bs, D = k_cache.shape
    _check(library().pa_copy_blocks(
        _ptr(k_cache), _ptr(v_cache), _ptr(block_mapping), block_mapping.shape[0], Hkv, D, bs, N,
        _dtype_code(k_cache), _ptr(err_flag), _stream(stream)), "pa_copy_blocks")


# ---------------------------------------------------------------------------
# prefix-deduplicated decode
# ---------------------------------------------------------------------------
@dataclass
class SharedPrefixGroups:
    """Groups of sequences that share their leading blocks (``pa_shared_prefix_plan``):
    group g's members are ``seqs[start[g]:start[g+1]]`` and share ``blocks[g]`` blocks."""
    seqs: np.ndarray
    start: np.ndarray
    blocks: np.ndarray

    @property
    def num_groups(self) -> int:
        return len(self.blocks)

    @property
    def num_listed(self) -> int:
        return len(self.seqs)

    def to(self, device="cuda"):
        """(seqs, start, blocks) as int32 device tensors."""
        return tuple(torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(device)
                     for a in (self.seqs, self.start, self.blocks))


def shared_prefix_plan(block_tables: np.ndarray, context_lens: np.ndarray,
                       min_shared_blocks: int = 1, tree: bool = False) -> SharedPrefixGroups:
    """Find the groups on the host (the library's planner; no device needed):
    one group per first block, or with ``tree`` groups chosen on the trie of
    block paths (``pa_shared_prefix_plan_tree``)."""
    bt = np.ascontiguousarray(block_tables, dtype=np.int32)
    cl = np.ascontiguousarray(context_lens, dtype=np.int32)
    S = int(cl.shape[0])
    if bt.ndim != 2 or bt.shape[0] != S:
        raise ValueError("block_tables must be [num_seqs][max_blocks_per_seq]")
    seqs = np.zeros(max(S, 1), dtype=np.int32)
    start = np.zeros(S + 1, dtype=np.int32)
    blocks = np.zeros(max(S, 1), dtype=np.int32)
    ng, nl = ctypes.c_int(0), ctypes.c_int(0)
    vp = ctypes.c_void_p
    fn = "pa_shared_prefix_plan_tree" if tree else "pa_shared_prefix_plan"
    _check(getattr(library(), fn)(
        vp(bt.ctypes.data), vp(cl.ctypes.data), S, int(bt.shape[1]), 16, int(min_shared_blocks),
        vp(seqs.ctypes.data), vp(start.ctypes.data), vp(blocks.ctypes.data), ctypes.byref(ng),
        ctypes.byref(nl)), fn)
    return SharedPrefixGroups(seqs[:nl.value].copy(), start[:ng.value + 1].copy(),
                              blocks[:ng.value].copy())


def shared_prefix_workspace_size(num_seqs: int, num_listed: int, num_q_heads: int,
                                 num_kv_heads: int, head_dim: int, max_blocks_per_seq: int,
                                 max_context_len: int, partition_size: int = 0,
                                 dtype: torch.dtype = torch.bfloat16) -> int:
    out = ctypes.c_size_t(0)
    _check(library().pa_shared_prefix_workspace_size(
        num_seqs, num_listed, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
        int(max_context_len), int(partition_size),
        PA_BF16 if dtype == torch.bfloat16 else PA_F32, ctypes.byref(out)),
        "pa_shared_prefix_workspace_size")
    return int(out.value)


def make_shared_prefix_workspace(num_seqs: int, num_listed: int, num_q_heads: int,
                                 num_kv_heads: int, head_dim: int, max_blocks_per_seq: int,
                                 max_context_len: int, partition_size: int = 0,
                                 dtype: torch.dtype = torch.bfloat16, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of the size ``pa_decode_shared_prefix`` needs."""
    n = shared_prefix_workspace_size(num_seqs, num_listed, num_q_heads, num_kv_heads, head_dim,
                                     max_blocks_per_seq, max_context_len, partition_size, dtype)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def decode_shared_prefix(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                         v_cache: torch.Tensor, block_tables: torch.Tensor,
                         context_lens: torch.Tensor, groups, *, scale: float,
                         max_context_len: int, workspace: torch.Tensor,
                         key: Optional[torch.Tensor] = None, value: Optional[torch.Tensor] = None,
                         partition_size: int = 0, err_flag: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """Decode that reads each group's shared blocks once; ``groups`` is the
    (seqs, start, blocks) device triple of :meth:`SharedPrefixGroups.to`.  With
    ``key``/``value`` the newest rows are also written, as in :func:`decode_append`."""
    seqs, start, blocks = groups
    S, Hq, D = q.shape
    N, Hkv, bs, _ = k_cache.shape
    _check(library().pa_decode_shared_prefix(
        _ptr(out), _ptr(q), _ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_tables), _ptr(context_lens), _ptr(seqs), _ptr(start), _ptr(blocks),
        int(blocks.numel()), int(seqs.numel()), S, Hq, Hkv, D, bs, block_tables.shape[1], N,
        int(max_context_len), float(scale), int(partition_size), _dtype_code(q), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(err_flag), _stream(stream)),
        "pa_decode_shared_prefix")
    return out
