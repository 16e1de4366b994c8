"""GB300-native (sm_103a) paged decode attention.

The computation lives in the CUDA library ``lib/libpagedattn.so`` behind the
C ABI of ``include/pa.h``.  This module only marshals PyTorch tensors (device
memory and the current CUDA stream) into those calls; there is no CPU or
PyTorch fallback - a missing library raises.

    reshape_and_cache(key, value, k_cache, v_cache, slot_mapping)
    decode(out, query, k_cache, v_cache, block_tables, context_lens, scale, ...)
    prefill(out, query, k_cache, v_cache, block_tables, context_lens, cu_seqlens_q, scale, ...)
    copy_blocks(k_cache, v_cache, block_mapping)
    decode_shared(out, query, k_cache, v_cache, block_tables, context_lens, cu_groups, shared_lens, scale, ...)
    quant_reshape_and_cache(key, value, k_cache, v_cache, k_scales, v_scales, slot_mapping)
    quant_gather(out_k, out_v, k_cache, v_cache, k_scales, v_scales, block_tables, cu_seqlens, ...)
    quant_decode(out, query, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale, ...)
    int4_reshape_and_cache, int4_gather, int4_decode: the same over caches of 4-bit codes
    update_tables(block_tables, context_lens, changes, free_blocks, free_count, slot_mapping, positions, cu_seqlens, ...)
    rope_and_cache(out_q, query, key, value, k_cache, v_cache, slot_mapping, positions, inv_freq, ...)

Cache layout: ``[num_blocks, block_size, num_kv_heads, head_dim]`` per layer
for K and for V ("LLM推理优化：vLLM PagedAttention深度解析与工程实践", §4.1).
Caches are float16 / bfloat16, or FP8 e4m3 codes (``torch.float8_e4m3fn`` or
``torch.uint8``) with per-tensor ``k_scale`` / ``v_scale``; the ``quant_*`` calls
keep int8 or e4m3 codes with a float32 scale per token and KV head,
``[num_blocks, block_size, num_kv_heads]``.  :func:`copy_blocks` and
:func:`swap_blocks` move such a cache as bytes: ``codes.view(torch.uint8)``, and
``scales.view(torch.uint8).view(NB, bs, Hkv, 4)``.  The ``int4_*`` calls keep two
codes to a byte, ``torch.uint8`` ``[NB, bs, Hkv, D/2]``, with a bfloat16 scale and zero
per 64 elements, ``[NB, Hkv, bs, D/64, 2]`` (heads before tokens).
"""
from __future__ import annotations

import ctypes
import functools
import math
import threading

from . import _lib
from ._lib import (FLAG_BAD_BLOCK_ID, FLAG_BAD_CONTEXT_LEN, FLAG_BAD_COPY_PAIR, FLAG_BAD_SLOT,
                   FLAG_NO_BLOCKS, FLAG_TIMEOUT, PA_BF16, PA_F16, PA_F32, PA_FP8_E4M3, PA_INT4, PA_INT8,
                   PagedAttentionError)

__all__ = ["reshape_and_cache", "decode", "decode_append", "prefill", "copy_blocks", "copy_blocks_layers", "swap_blocks", "decode_workspace_size",
           "decode_partition_size", "DecodeWorkspace", "new_err_flag", "read_err_flag",
           "quant_reshape_and_cache", "quant_gather", "quant_decode", "quant_decode_workspace_size", "decode_shared",
           "update_tables", "rope_and_cache", "rope_frequencies", "FLAG_NO_BLOCKS",
           "int4_reshape_and_cache", "int4_gather", "int4_decode", "int4_decode_workspace_size",
           "decode_shared_workspace_size", "PagedAttentionError", "FLAG_BAD_SLOT", "FLAG_BAD_BLOCK_ID", "FLAG_BAD_CONTEXT_LEN",
           "FLAG_BAD_COPY_PAIR", "FLAG_TIMEOUT", "library_path", "StepGraph"]


def library_path() -> str:
    return _lib.lib_path()


def _torch():
    import torch
    return torch


def _dtype_code(t, allow_f32=False) -> int:
    torch = _torch()
    if t.dtype == torch.float16:
        return PA_F16
    if t.dtype == torch.bfloat16:
        return PA_BF16
    if allow_f32 and t.dtype == torch.float32:
        return PA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _cache_code(t) -> int:
    torch = _torch()
    if t.dtype in (torch.uint8, getattr(torch, "float8_e4m3fn", None)):
        return PA_FP8_E4M3
    return _dtype_code(t)


def _need(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _cuda_contig(name, t):
    _need(t.is_cuda, f"{name} must be a CUDA tensor")
    _need(t.is_contiguous(), f"{name} must be contiguous")


def _stream(device) -> ctypes.c_void_p:
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def new_err_flag(device=None):
    """A zeroed device int32 that kernels OR their PA_FLAG_* bits into."""
    torch = _torch()
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def read_err_flag(err_flag, clear: bool = True) -> int:
    """Synchronise the current stream and return (optionally clearing) the flag bits."""
    lib = _lib.load()
    out = ctypes.c_int(0)
    st = lib.pa_check_err_flag(_ptr(err_flag), int(clear), ctypes.byref(out), _stream(err_flag.device))
    if st not in (_lib.PA_OK, _lib.PA_ERR_DEVICE_BOUNDS):
        _lib.check(st, "pa_check_err_flag")
    return int(out.value)


def reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, err_flag=None,
                      k_scale: float = 1.0, v_scale: float = 1.0) -> None:
    """Write key/value rows [T, Hkv, D] into cache slots (slot < 0: skip);
    an FP8 cache receives e4m3(x / scale)."""
    for n, t in (("key", key), ("value", value), ("k_cache", k_cache), ("v_cache", v_cache),
                 ("slot_mapping", slot_mapping)):
        _cuda_contig(n, t)
    torch = _torch()
    _need(key.dim() == 3 and value.shape == key.shape, "key/value must be [T, Hkv, D]")
    _need(k_cache.dim() == 4 and v_cache.shape == k_cache.shape, "caches must be [NB, bs, Hkv, D]")
    _need(k_cache.shape[2:] == key.shape[1:], "cache and key head shapes differ")
    _need(key.dtype == value.dtype and k_cache.dtype == v_cache.dtype, "dtype mismatch")
    _need(slot_mapping.dtype == torch.int64 and slot_mapping.numel() == key.shape[0],
          "slot_mapping must be int64 [T]")
    nb, bs, hkv, d = k_cache.shape
    st = _lib.load().pa_reshape_and_cache(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
                                          _ptr(slot_mapping), key.shape[0], nb, bs, hkv, d,
                                          _dtype_code(key), _cache_code(k_cache), float(k_scale),
                                          float(v_scale), _ptr(err_flag), _stream(key.device))
    _lib.check(st, "pa_reshape_and_cache")


def copy_blocks(k_cache, v_cache, block_mapping, err_flag=None) -> None:
    """Copy whole blocks for each (src, dst) row of block_mapping [P, 2] int64."""
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache), ("block_mapping", block_mapping)):
        _cuda_contig(n, t)
    torch = _torch()
    _need(block_mapping.dtype == torch.int64 and block_mapping.dim() == 2 and block_mapping.shape[1] == 2,
          "block_mapping must be int64 [P, 2]")
    _need(k_cache.shape == v_cache.shape and k_cache.dtype == v_cache.dtype, "cache mismatch")
    nb, bs, hkv, d = k_cache.shape
    st = _lib.load().pa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(block_mapping),
                                    block_mapping.shape[0], nb, bs, hkv, d, _cache_code(k_cache),
                                    _ptr(err_flag), _stream(k_cache.device))
    _lib.check(st, "pa_copy_blocks")


def copy_blocks_layers(kv_cache, block_mapping, err_flag=None) -> None:
    """copy_blocks for every layer of a model's cache
    ``kv_cache`` [layers, 2, NB, bs, Hkv, D] (K at [l][0], V at [l][1]), one launch."""
    for n, t in (("kv_cache", kv_cache), ("block_mapping", block_mapping)):
        _cuda_contig(n, t)
    torch = _torch()
    _need(kv_cache.dim() == 6 and kv_cache.shape[1] == 2, "kv_cache must be [layers, 2, NB, bs, Hkv, D]")
    _need(block_mapping.dtype == torch.int64 and block_mapping.dim() == 2 and block_mapping.shape[1] == 2,
          "block_mapping must be int64 [P, 2]")
    layers, _, nb, bs, hkv, d = kv_cache.shape
    st = _lib.load().pa_copy_blocks_layers(_ptr(kv_cache), layers, _ptr(block_mapping), block_mapping.shape[0],
                                           nb, bs, hkv, d, _cache_code(kv_cache), _ptr(err_flag),
                                           _stream(kv_cache.device))
    _lib.check(st, "pa_copy_blocks_layers")


def swap_blocks(src_k, src_v, dst_k, dst_v, block_mapping, err_flag=None) -> None:
    """Copy whole blocks src -> dst between two caches (for swap-mode
    preemption); either cache may be a pinned host tensor (``pin_memory()``),
    the other a CUDA tensor.  ``block_mapping`` [P, 2] int64 on the GPU."""
    torch = _torch()
    for n, t in (("src_k", src_k), ("src_v", src_v), ("dst_k", dst_k), ("dst_v", dst_v)):
        _need(t.is_contiguous(), f"{n} must be contiguous")
        _need(t.is_cuda or t.is_pinned(), f"{n} must be a CUDA tensor or pinned host memory")
    _cuda_contig("block_mapping", block_mapping)
    _need(block_mapping.dtype == torch.int64 and block_mapping.dim() == 2 and block_mapping.shape[1] == 2,
          "block_mapping must be int64 [P, 2]")
    _need(src_k.shape[1:] == dst_k.shape[1:] and src_k.dtype == dst_k.dtype, "cache shapes differ")
    _need(src_v.shape == src_k.shape and dst_v.shape == dst_k.shape, "K and V caches differ")
    nb_src, bs, hkv, d = src_k.shape
    device = block_mapping.device
    st = _lib.load().pa_swap_blocks(_ptr(src_k), _ptr(src_v), _ptr(dst_k), _ptr(dst_v), _ptr(block_mapping),
                                    block_mapping.shape[0], nb_src, dst_k.shape[0], bs, hkv, d,
                                    _cache_code(src_k), _ptr(err_flag), _stream(device))
    _lib.check(st, "pa_swap_blocks")


def decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                          max_context_len, partition_size=0) -> int:
    n = _lib.load().pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                             max_context_len, partition_size)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("arguments rejected by pa_decode_workspace_size")
    return int(n)


def decode_partition_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                          max_context_len, partition_size=0) -> int:
    return int(_lib.load().pa_decode_partition_size(num_seqs, num_heads, num_kv_heads, head_dim,
                                                    block_size, max_context_len, partition_size))


class DecodeWorkspace:
    """A device workspace for pa_decode, grown on demand (no initial contents
    are needed).

    One instance must not serve two decode calls that can overlap on the GPU
    (the default per-(device, stream) instances used by :func:`decode` never do).
    """

    def __init__(self, device=None):
        self.device = device
        self.buf = None

    def get(self, nbytes: int, layout=None):
        """A buffer of at least ``nbytes`` bytes (None when nothing is needed)."""
        torch = _torch()
        if nbytes == 0:
            return None
        if self.buf is None or self.buf.numel() < nbytes:
            if self.buf is not None:
                # allocated on another stream perhaps, which may have its memory back once
                # this one is past the calls that used it
                self.buf.record_stream(torch.cuda.current_stream(self.buf.device))
            self.buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device or "cuda")
        return self.buf


_default_ws: dict = {}


def decode(out, query, k_cache, v_cache, block_tables, context_lens, scale: float,
           max_context_len: int | None = None, partition_size: int = 0, workspace=None,
           err_flag=None, k_scale: float = 1.0, v_scale: float = 1.0) -> None:
    """Paged decode attention into ``out`` [B, Hq, D] (f16, bf16 or f32).

    ``max_context_len`` is a host-side bound on ``context_lens`` (defaults to
    the block-table width times the block size)."""
    torch = _torch()
    for n, t in (("out", out), ("query", query), ("k_cache", k_cache), ("v_cache", v_cache),
                 ("block_tables", block_tables), ("context_lens", context_lens)):
        _cuda_contig(n, t)
    _need(query.dim() == 3 and out.shape == query.shape, "query/out must be [B, Hq, D]")
    _need(k_cache.dim() == 4 and v_cache.shape == k_cache.shape, "caches must be [NB, bs, Hkv, D]")
    _need(k_cache.dtype == v_cache.dtype, "K and V caches must share a dtype")
    _need(block_tables.dtype == torch.int32 and block_tables.dim() == 2 and
          block_tables.shape[0] == query.shape[0], "block_tables must be int32 [B, maxNB]")
    _need(context_lens.dtype == torch.int32 and context_lens.numel() == query.shape[0],
          "context_lens must be int32 [B]")
    B, Hq, D = query.shape
    nb, bs, hkv, d2 = k_cache.shape
    _need(d2 == D, "head_dim mismatch")
    maxnb = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = maxnb * bs
    ws_bytes = decode_workspace_size(B, Hq, hkv, D, bs, max_context_len, partition_size)
    if workspace is None:
        key = (query.device.index, torch.cuda.current_stream(query.device).cuda_stream)
        workspace = _default_ws.setdefault(key, DecodeWorkspace(query.device))
    layout = (B, Hq, hkv, D, bs, int(max_context_len), int(partition_size))
    buf = workspace.get(ws_bytes, layout) if isinstance(workspace, DecodeWorkspace) else workspace
    nbytes = 0 if buf is None else buf.numel() * buf.element_size()
    st = _lib.load().pa_decode(_ptr(out), _dtype_code(out, allow_f32=True), _ptr(query), _dtype_code(query),
                               _ptr(k_cache), _ptr(v_cache), _cache_code(k_cache), float(k_scale),
                               float(v_scale), _ptr(block_tables),
                               maxnb, _ptr(context_lens), int(max_context_len), B, Hq, hkv, D, bs, nb,
                               float(scale), int(partition_size), _ptr(buf), nbytes, _ptr(err_flag),
                               _stream(query.device))
    _lib.check(st, "pa_decode")


def decode_append(out, query, key, value, k_cache, v_cache, block_tables, context_lens, scale: float,
                  max_context_len: int | None = None, partition_size: int = 0, workspace=None,
                  err_flag=None, k_scale: float = 1.0, v_scale: float = 1.0) -> None:
    """reshape_and_cache of each sequence's new token (position context_lens[s] - 1,
    rows ``key``/``value`` [B, Hkv, D]) fused with :func:`decode`, one launch."""
    torch = _torch()
    for n, t in (("out", out), ("query", query), ("key", key), ("value", value), ("k_cache", k_cache),
                 ("v_cache", v_cache), ("block_tables", block_tables), ("context_lens", context_lens)):
        _cuda_contig(n, t)
    _need(query.dim() == 3 and out.shape == query.shape, "query/out must be [B, Hq, D]")
    _need(k_cache.dim() == 4 and v_cache.shape == k_cache.shape and k_cache.dtype == v_cache.dtype,
          "caches must be [NB, bs, Hkv, D] of one dtype")
    B, Hq, D = query.shape
    nb, bs, hkv, d2 = k_cache.shape
    _need(d2 == D and key.shape == (B, hkv, D) and value.shape == key.shape, "key/value must be [B, Hkv, D]")
    _need(key.dtype == value.dtype == query.dtype, "key/value must have the query's dtype")
    _need(block_tables.dtype == torch.int32 and block_tables.dim() == 2 and block_tables.shape[0] == B,
          "block_tables must be int32 [B, maxNB]")
    _need(context_lens.dtype == torch.int32 and context_lens.numel() == B, "context_lens must be int32 [B]")
    maxnb = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = maxnb * bs
    ws_bytes = decode_workspace_size(B, Hq, hkv, D, bs, max_context_len, partition_size)
    if workspace is None:
        wkey = (query.device.index, torch.cuda.current_stream(query.device).cuda_stream)
        workspace = _default_ws.setdefault(wkey, DecodeWorkspace(query.device))
    buf = workspace.get(ws_bytes) if isinstance(workspace, DecodeWorkspace) else workspace
    nbytes = 0 if buf is None else buf.numel() * buf.element_size()
    st = _lib.load().pa_decode_append(_ptr(out), _dtype_code(out, allow_f32=True), _ptr(query),
                                      _dtype_code(query), _ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
                                      _cache_code(k_cache), float(k_scale), float(v_scale), _ptr(block_tables),
                                      maxnb, _ptr(context_lens), int(max_context_len), B, Hq, hkv, D, bs, nb,
                                      float(scale), int(partition_size), _ptr(buf), nbytes, _ptr(err_flag),
                                      _stream(query.device))
    _lib.check(st, "pa_decode_append")


def prefill(out, query, k_cache, v_cache, block_tables, context_lens, cu_seqlens_q, scale: float,
            max_q_len: int, err_flag=None) -> None:
    """Causal attention of each sequence's newest tokens over its paged context
    into ``out`` [T, Hq, D] (f16, bf16 or f32).

    Sequence s owns query rows ``cu_seqlens_q[s] .. cu_seqlens_q[s+1]-1`` (int32
    [B+1] on the GPU); ``context_lens[s]`` counts all its tokens, new ones
    included (their K/V rows already written with :func:`reshape_and_cache`).
    ``max_q_len`` is a host-side bound on every sequence's new-token count."""
    torch = _torch()
    for n, t in (("out", out), ("query", query), ("k_cache", k_cache), ("v_cache", v_cache),
                 ("block_tables", block_tables), ("context_lens", context_lens),
                 ("cu_seqlens_q", cu_seqlens_q)):
        _cuda_contig(n, t)
    _need(query.dim() == 3 and out.shape == query.shape, "query/out must be [T, Hq, D]")
    _need(k_cache.dim() == 4 and v_cache.shape == k_cache.shape and k_cache.dtype == v_cache.dtype,
          "caches must be [NB, bs, Hkv, D] of one dtype")
    _need(k_cache.dtype == query.dtype, "caches must have the query's dtype")
    B = context_lens.numel()
    _need(context_lens.dtype == torch.int32, "context_lens must be int32 [B]")
    _need(cu_seqlens_q.dtype == torch.int32 and cu_seqlens_q.numel() == B + 1, "cu_seqlens_q must be int32 [B+1]")
    _need(block_tables.dtype == torch.int32 and block_tables.dim() == 2 and block_tables.shape[0] == B,
          "block_tables must be int32 [B, maxNB]")
    T, Hq, D = query.shape
    nb, bs, hkv, d2 = k_cache.shape
    _need(d2 == D, "head_dim mismatch")
    st = _lib.load().pa_prefill(_ptr(out), _dtype_code(out, allow_f32=True), _ptr(query), _ptr(k_cache),
                                _ptr(v_cache), _dtype_code(query), _ptr(block_tables), block_tables.shape[1],
                                _ptr(context_lens), _ptr(cu_seqlens_q), B, T, int(max_q_len), Hq, hkv, D, bs,
                                nb, float(scale), _ptr(err_flag), _stream(query.device))
    _lib.check(st, "pa_prefill")


# ------------------------- quantised cache, and decode with shared prefixes
#
# These calls are made once per layer and step on small tensors, where the
# marshalling itself counts (16 us of a 21 us write of four rows before it was
# written this way): each looks its tensors over in one expression and explains
# a refusal only when that fails.

class _Codes(dict):
    """pa_dtype codes by torch dtype; others are refused."""

    def __missing__(self, dtype):
        raise TypeError(f"unsupported dtype {dtype}")


class _Runtime:
    """What the calls below need of torch and the library, looked up once."""

    def __init__(self):
        torch = _torch()
        self.lib = _lib.load()
        self.half = _Codes({torch.float16: PA_F16, torch.bfloat16: PA_BF16})
        self.out = _Codes({**self.half, torch.float32: PA_F32})
        self.codes = _Codes({torch.int8: PA_INT8, torch.uint8: PA_FP8_E4M3, torch.float8_e4m3fn: PA_FP8_E4M3})
        self.b16, self.f64 = torch.bfloat16, torch.float64
        self.f32, self.i32, self.i64, self.u8 = torch.float32, torch.int32, torch.int64, torch.uint8
        self.current_device = torch._C._cuda_getDevice      # (without the first-use checks: the tensors exist)
        self.capturing = torch.cuda.is_current_stream_capturing
        self.stream = torch._C._cuda_getCurrentRawStream
        self.empty = torch.empty


_rt = None


def _runtime():
    global _rt
    if _rt is None:
        _rt = _Runtime()
    return _rt


def _refuse(tensors, message=None):
    """Raise for the first of (name, tensor) that is not contiguous on the current
    CUDA device, else with ``message``."""
    for n, t in tensors:
        _cuda_contig(n, t)
        _need(t.get_device() == _runtime().current_device(), f"{n} must be on the current CUDA device")
    raise ValueError(message or "tensors must be on the current CUDA device")


def _flag(err_flag, dev: int):
    if err_flag.get_device() != dev or err_flag.element_size() != 4:
        raise ValueError("err_flag must be an int32 tensor on the device of the others (new_err_flag)")
    return err_flag.data_ptr()


_thread_ws = threading.local()       # .by_stream: {(device, stream): DecodeWorkspace} of one thread


def _scratch(rt, workspace, nbytes: int, dev: int, stream: int):
    """The workspace of one call: the caller's, the calling thread's default one for
    the current stream (a call is several launches, between which another thread's
    may come), kept until the thread ends, or, while a graph is captured, one of the graph's own (so that
    graphs never share one and none is replaced by a larger one later)."""
    if nbytes == 0:
        return None
    if workspace is None:
        if rt.capturing():
            return rt.empty(nbytes, dtype=rt.u8, device=dev)
        try:
            workspace = _thread_ws.by_stream.get((dev, stream))
        except AttributeError:
            _thread_ws.by_stream = {}
        if workspace is None:
            workspace = _thread_ws.by_stream[dev, stream] = DecodeWorkspace(_torch().device("cuda", dev))
    if isinstance(workspace, DecodeWorkspace):
        workspace = workspace.get(nbytes)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse((("workspace", workspace),))
    return workspace


def quant_reshape_and_cache(key, value, k_cache, v_cache, k_scales, v_scales, slot_mapping, err_flag=None) -> None:
    """Quantise key/value rows [T, Hkv, D] (f16 or bf16) into cache slots
    (slot < 0: skip), one scale per token and KV head.

    The caches' dtype chooses the codes: ``torch.int8``, or e4m3 for
    ``torch.float8_e4m3fn`` / ``torch.uint8``.  key and value may be slices along
    the last two dimensions of a wider tensor (a token's rows dense, any token
    stride that is a multiple of 8 elements)."""
    rt = _rt or _runtime()
    dev, shape, cache = key.get_device(), key.shape, k_cache.shape
    if (dev != rt.current_device() or value.get_device() != dev or k_cache.get_device() != dev or
            v_cache.get_device() != dev or k_scales.get_device() != dev or v_scales.get_device() != dev or
            slot_mapping.get_device() != dev or not k_cache.is_contiguous() or not v_cache.is_contiguous() or
            not k_scales.is_contiguous() or not v_scales.is_contiguous() or not slot_mapping.is_contiguous()):
        _refuse((("k_cache", k_cache), ("v_cache", v_cache), ("k_scales", k_scales), ("v_scales", v_scales),
                 ("slot_mapping", slot_mapping)), "key and value must be on the device of the caches")
    if len(shape) != 3 or value.shape != shape or value.dtype != key.dtype:
        raise ValueError("key/value must be [T, Hkv, D] of one dtype")
    T, hkv, d = shape
    if len(cache) != 4 or v_cache.shape != cache or v_cache.dtype != k_cache.dtype or cache[2] != hkv or cache[3] != d:
        raise ValueError("caches must be [NB, bs, Hkv, D] of one dtype, with the rows' heads")
    nb, bs = cache[0], cache[1]
    rows = (nb, bs, hkv)
    if k_scales.shape != rows or v_scales.shape != rows or k_scales.dtype != rt.f32 or v_scales.dtype != rt.f32:
        raise ValueError("scales must be float32 [NB, bs, Hkv]")
    if slot_mapping.dtype != rt.i64 or slot_mapping.numel() != T:
        raise ValueError("slot_mapping must be int64 [T]")
    ks, vs = key.stride(), value.stride()
    if ks[2] != 1 or vs[2] != 1 or (hkv != 1 and (ks[1] != d or vs[1] != d)):
        raise ValueError("key/value: the rows of one token must be dense")
    one = T <= 1
    st = rt.lib.pa_quant_reshape_and_cache(
        key.data_ptr(), value.data_ptr(), hkv * d if one else ks[0], hkv * d if one else vs[0], k_cache.data_ptr(),
        v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), slot_mapping.data_ptr(), T, nb, bs, hkv,
        d, rt.half[key.dtype], rt.codes[k_cache.dtype],
        None if err_flag is None else _flag(err_flag, dev), rt.stream(dev))
    if st:
        _lib.check(st, "pa_quant_reshape_and_cache")


def quant_gather(out_k, out_v, k_cache, v_cache, k_scales, v_scales, block_tables, cu_seqlens, seq_starts=None,
                 err_flag=None) -> None:
    """Read a quantised cache back: row ``cu_seqlens[s] + i`` of out_k/out_v
    [T, Hkv, D] (f16, bf16 or f32) becomes sequence s's position
    ``seq_starts[s] + i`` (``seq_starts`` None: 0).  Rows from ``cu_seqlens[-1]``
    on are left as they were."""
    rt = _rt or _runtime()
    dev, cache, shape, table = out_k.get_device(), k_cache.shape, out_k.shape, block_tables.shape
    if (dev != rt.current_device() or out_v.get_device() != dev or k_cache.get_device() != dev or
            v_cache.get_device() != dev or k_scales.get_device() != dev or v_scales.get_device() != dev or
            block_tables.get_device() != dev or cu_seqlens.get_device() != dev or not out_k.is_contiguous() or
            not out_v.is_contiguous() or not k_cache.is_contiguous() or not v_cache.is_contiguous() or
            not k_scales.is_contiguous() or not v_scales.is_contiguous() or not block_tables.is_contiguous() or
            not cu_seqlens.is_contiguous()):
        _refuse((("out_k", out_k), ("out_v", out_v), ("k_cache", k_cache), ("v_cache", v_cache), ("k_scales", k_scales),
                 ("v_scales", v_scales), ("block_tables", block_tables), ("cu_seqlens", cu_seqlens)))
    if len(cache) != 4 or v_cache.shape != cache or v_cache.dtype != k_cache.dtype:
        raise ValueError("caches must be [NB, bs, Hkv, D] of one dtype")
    nb, bs, hkv, d = cache
    rows = (nb, bs, hkv)
    if k_scales.shape != rows or v_scales.shape != rows or k_scales.dtype != rt.f32 or v_scales.dtype != rt.f32:
        raise ValueError("scales must be float32 [NB, bs, Hkv]")
    if len(shape) != 3 or out_v.shape != shape or out_v.dtype != out_k.dtype or shape[1] != hkv or shape[2] != d:
        raise ValueError("out_k/out_v must be [T, Hkv, D] of one dtype")
    if len(table) != 2 or block_tables.dtype != rt.i32:
        raise ValueError("block_tables must be int32 [B, maxNB]")
    B = table[0]
    if cu_seqlens.dtype != rt.i32 or cu_seqlens.numel() != B + 1:
        raise ValueError("cu_seqlens must be int32 [B+1]")
    if seq_starts is not None:
        if seq_starts.get_device() != dev or not seq_starts.is_contiguous():
            _refuse((("seq_starts", seq_starts),))
        if seq_starts.dtype != rt.i32 or seq_starts.numel() != B:
            raise ValueError("seq_starts must be int32 [B]")
    st = rt.lib.pa_quant_gather(
        out_k.data_ptr(), out_v.data_ptr(), rt.out[out_k.dtype], k_cache.data_ptr(), v_cache.data_ptr(),
        rt.codes[k_cache.dtype], k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(), table[1],
        cu_seqlens.data_ptr(), None if seq_starts is None else seq_starts.data_ptr(), B, shape[0], hkv, d, bs,
        nb, None if err_flag is None else _flag(err_flag, dev), rt.stream(dev))
    if st:
        _lib.check(st, "pa_quant_gather")


@functools.lru_cache(maxsize=1024)
def quant_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len,
                                partition_size=0) -> int:
    n = _lib.load().pa_quant_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                   max_context_len, partition_size)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("arguments rejected by pa_quant_decode_workspace_size")
    return n


def _decode_shapes(rt, out, query, cache, v_cache, block_tables, context_lens):
    shape, table = query.shape, block_tables.shape
    if len(shape) != 3 or out.shape != shape:
        raise ValueError("query/out must be [B, Hq, D]")
    if len(cache) != 4 or v_cache.shape != cache or cache[3] != shape[2]:
        raise ValueError("caches must be [NB, bs, Hkv, D] with the query's D")
    if len(table) != 2 or table[0] != shape[0] or block_tables.dtype != rt.i32:
        raise ValueError("block_tables must be int32 [B, maxNB]")
    if context_lens.dtype != rt.i32 or context_lens.numel() != shape[0]:
        raise ValueError("context_lens must be int32 [B]")


def quant_decode(out, query, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale: float,
                 max_context_len: int | None = None, partition_size: int = 0, workspace=None, err_flag=None) -> None:
    """:func:`decode` over a quantised cache written by :func:`quant_reshape_and_cache`."""
    rt = _rt or _runtime()
    dev, cache = query.get_device(), k_cache.shape
    if (dev != rt.current_device() or out.get_device() != dev or k_cache.get_device() != dev or
            v_cache.get_device() != dev or k_scales.get_device() != dev or v_scales.get_device() != dev or
            block_tables.get_device() != dev or context_lens.get_device() != dev or not query.is_contiguous() or
            not out.is_contiguous() or not k_cache.is_contiguous() or not v_cache.is_contiguous() or
            not k_scales.is_contiguous() or not v_scales.is_contiguous() or not block_tables.is_contiguous() or
            not context_lens.is_contiguous()):
        _refuse((("query", query), ("out", out), ("k_cache", k_cache), ("v_cache", v_cache), ("k_scales", k_scales),
                 ("v_scales", v_scales), ("block_tables", block_tables), ("context_lens", context_lens)))
    _decode_shapes(rt, out, query, cache, v_cache, block_tables, context_lens)
    if v_cache.dtype != k_cache.dtype:
        raise ValueError("K and V caches must share a dtype")
    B, Hq, D = query.shape
    nb, bs, hkv, _ = cache
    rows = (nb, bs, hkv)
    if k_scales.shape != rows or v_scales.shape != rows or k_scales.dtype != rt.f32 or v_scales.dtype != rt.f32:
        raise ValueError("scales must be float32 [NB, bs, Hkv]")
    maxnb = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = maxnb * bs
    stream = rt.stream(dev)
    buf = _scratch(rt, workspace, quant_decode_workspace_size(B, Hq, hkv, D, bs, max_context_len, partition_size), dev,
                   stream)
    st = rt.lib.pa_quant_decode(
        out.data_ptr(), rt.out[out.dtype], query.data_ptr(), rt.half[query.dtype],
        k_cache.data_ptr(), v_cache.data_ptr(), rt.codes[k_cache.dtype], k_scales.data_ptr(),
        v_scales.data_ptr(), block_tables.data_ptr(), maxnb, context_lens.data_ptr(), max_context_len, B, Hq, hkv, D, bs,
        nb, scale, partition_size, None if buf is None else buf.data_ptr(), 0 if buf is None else buf.nbytes,
        None if err_flag is None else _flag(err_flag, dev), stream)
    if st:
        _lib.check(st, "pa_quant_decode")


def _int4_cache(rt, k_cache, v_cache, k_scales, v_scales, d: int):
    """(num_blocks, block_size, num_kv_heads) of a 4-bit cache for rows of d elements."""
    shape = k_cache.shape
    if (len(shape) != 4 or v_cache.shape != shape or 2 * shape[3] != d or k_cache.dtype != rt.u8 or
            v_cache.dtype != rt.u8):
        raise ValueError("caches must be uint8 [NB, bs, Hkv, D/2]")
    nb, bs, hkv, _ = shape
    words = (nb, hkv, bs, d // 64, 2)
    if k_scales.shape != words or v_scales.shape != words or k_scales.dtype != rt.b16 or v_scales.dtype != rt.b16:
        raise ValueError("scales must be bfloat16 [NB, Hkv, bs, D/64, 2]")
    return nb, bs, hkv


def int4_reshape_and_cache(key, value, k_cache, v_cache, k_scales, v_scales, slot_mapping, err_flag=None) -> None:
    """Write key/value rows [T, Hkv, D] (f16 or bf16) into cache slots (slot < 0:
    skip) as 4-bit codes, a scale and a zero per 64 elements.

    key and value may be slices of a wider tensor, as for :func:`quant_reshape_and_cache`."""
    rt = _rt or _runtime()
    dev, shape = key.get_device(), key.shape
    if (dev != rt.current_device() or value.get_device() != dev or k_cache.get_device() != dev or
            v_cache.get_device() != dev or k_scales.get_device() != dev or v_scales.get_device() != dev or
            slot_mapping.get_device() != dev or not k_cache.is_contiguous() or not v_cache.is_contiguous() or
            not k_scales.is_contiguous() or not v_scales.is_contiguous() or not slot_mapping.is_contiguous()):
        _refuse((("k_cache", k_cache), ("v_cache", v_cache), ("k_scales", k_scales), ("v_scales", v_scales),
                 ("slot_mapping", slot_mapping)), "key and value must be on the device of the caches")
    if len(shape) != 3 or value.shape != shape or value.dtype != key.dtype:
        raise ValueError("key/value must be [T, Hkv, D] of one dtype")
    T, hkv, d = shape
    nb, bs, heads = _int4_cache(rt, k_cache, v_cache, k_scales, v_scales, d)
    if heads != hkv:
        raise ValueError("cache and key heads differ")
    if slot_mapping.dtype != rt.i64 or slot_mapping.numel() != T:
        raise ValueError("slot_mapping must be int64 [T]")
    ks, vs = key.stride(), value.stride()
    if ks[2] != 1 or vs[2] != 1 or (hkv != 1 and (ks[1] != d or vs[1] != d)):
        raise ValueError("key/value: the rows of one token must be dense")
    one = T <= 1
    st = rt.lib.pa_int4_reshape_and_cache(
        key.data_ptr(), value.data_ptr(), hkv * d if one else ks[0], hkv * d if one else vs[0], k_cache.data_ptr(),
        v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), slot_mapping.data_ptr(), T, nb, bs, hkv,
        d, rt.half[key.dtype], None if err_flag is None else _flag(err_flag, dev), rt.stream(dev))
    if st:
        _lib.check(st, "pa_int4_reshape_and_cache")


def int4_gather(out_k, out_v, k_cache, v_cache, k_scales, v_scales, block_tables, cu_seqlens, seq_starts=None,
                err_flag=None) -> None:
    """:func:`quant_gather` from a 4-bit cache written by :func:`int4_reshape_and_cache`."""
    rt = _rt or _runtime()
    dev, shape, table = out_k.get_device(), out_k.shape, block_tables.shape
    if (dev != rt.current_device() or out_v.get_device() != dev or k_cache.get_device() != dev or
            v_cache.get_device() != dev or k_scales.get_device() != dev or v_scales.get_device() != dev or
            block_tables.get_device() != dev or cu_seqlens.get_device() != dev or not out_k.is_contiguous() or
            not out_v.is_contiguous() or not k_cache.is_contiguous() or not v_cache.is_contiguous() or
            not k_scales.is_contiguous() or not v_scales.is_contiguous() or not block_tables.is_contiguous() or
            not cu_seqlens.is_contiguous()):
        _refuse((("out_k", out_k), ("out_v", out_v), ("k_cache", k_cache), ("v_cache", v_cache), ("k_scales", k_scales),
                 ("v_scales", v_scales), ("block_tables", block_tables), ("cu_seqlens", cu_seqlens)))
    if len(shape) != 3 or out_v.shape != shape or out_v.dtype != out_k.dtype:
        raise ValueError("out_k/out_v must be [T, Hkv, D] of one dtype")
    d = shape[2]
    nb, bs, hkv = _int4_cache(rt, k_cache, v_cache, k_scales, v_scales, d)
    if shape[1] != hkv:
        raise ValueError("cache and out_k heads differ")
    if len(table) != 2 or block_tables.dtype != rt.i32:
        raise ValueError("block_tables must be int32 [B, maxNB]")
    B = table[0]
    if cu_seqlens.dtype != rt.i32 or cu_seqlens.numel() != B + 1:
        raise ValueError("cu_seqlens must be int32 [B+1]")
    if seq_starts is not None:
        if seq_starts.get_device() != dev or not seq_starts.is_contiguous():
            _refuse((("seq_starts", seq_starts),))
        if seq_starts.dtype != rt.i32 or seq_starts.numel() != B:
            raise ValueError("seq_starts must be int32 [B]")
    st = rt.lib.pa_int4_gather(
        out_k.data_ptr(), out_v.data_ptr(), rt.out[out_k.dtype], k_cache.data_ptr(), v_cache.data_ptr(),
        k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(), table[1], cu_seqlens.data_ptr(),
        None if seq_starts is None else seq_starts.data_ptr(), B, shape[0], hkv, d, bs, nb,
        None if err_flag is None else _flag(err_flag, dev), rt.stream(dev))
    if st:
        _lib.check(st, "pa_int4_gather")


@functools.lru_cache(maxsize=1024)
def int4_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len,
                               partition_size=0) -> int:
    n = _lib.load().pa_int4_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                  max_context_len, partition_size)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("arguments rejected by pa_int4_decode_workspace_size")
    return n


def int4_decode(out, query, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale: float,
                max_context_len: int | None = None, partition_size: int = 0, workspace=None, err_flag=None) -> None:
    """:func:`decode` over a 4-bit cache written by :func:`int4_reshape_and_cache`."""
    rt = _rt or _runtime()
    dev, shape, table = query.get_device(), query.shape, block_tables.shape
    if (dev != rt.current_device() or out.get_device() != dev or k_cache.get_device() != dev or
            v_cache.get_device() != dev or k_scales.get_device() != dev or v_scales.get_device() != dev or
            block_tables.get_device() != dev or context_lens.get_device() != dev or not query.is_contiguous() or
            not out.is_contiguous() or not k_cache.is_contiguous() or not v_cache.is_contiguous() or
            not k_scales.is_contiguous() or not v_scales.is_contiguous() or not block_tables.is_contiguous() or
            not context_lens.is_contiguous()):
        _refuse((("query", query), ("out", out), ("k_cache", k_cache), ("v_cache", v_cache), ("k_scales", k_scales),
                 ("v_scales", v_scales), ("block_tables", block_tables), ("context_lens", context_lens)))
    if len(shape) != 3 or out.shape != shape:
        raise ValueError("query/out must be [B, Hq, D]")
    B, Hq, D = shape
    nb, bs, hkv = _int4_cache(rt, k_cache, v_cache, k_scales, v_scales, D)
    if len(table) != 2 or table[0] != B or block_tables.dtype != rt.i32:
        raise ValueError("block_tables must be int32 [B, maxNB]")
    if context_lens.dtype != rt.i32 or context_lens.numel() != B:
        raise ValueError("context_lens must be int32 [B]")
    maxnb = table[1]
    if max_context_len is None:
        max_context_len = maxnb * bs
    stream = rt.stream(dev)
    buf = _scratch(rt, workspace, int4_decode_workspace_size(B, Hq, hkv, D, bs, max_context_len, partition_size), dev,
                   stream)
    st = rt.lib.pa_int4_decode(
        out.data_ptr(), rt.out[out.dtype], query.data_ptr(), rt.half[query.dtype], k_cache.data_ptr(),
        v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(), maxnb,
        context_lens.data_ptr(), max_context_len, B, Hq, hkv, D, bs, nb, scale, partition_size,
        None if buf is None else buf.data_ptr(), 0 if buf is None else buf.nbytes,
        None if err_flag is None else _flag(err_flag, dev), stream)
    if st:
        _lib.check(st, "pa_int4_decode")


# ------------------------------------- a step's bookkeeping and its rotation

def update_tables(block_tables, context_lens, changes, free_blocks, free_count, slot_mapping, positions, cu_seqlens,
                  block_size: int, num_blocks: int | None = None, out_lens=None, out_free_count=None, err_flag=None) -> None:
    """Bring a batch's block tables and lengths up to date on the GPU.

    Sequence s grows by ``changes[s]`` tokens (int32 [B]) or, for a negative change,
    drops its newest ones (all of them: it ends); its blocks come from and go back to
    the stack ``free_blocks`` (int32 [capacity], the first ``free_count`` (int32 [1]) of
    them free, the last of those taken next).  ``block_tables`` (int32 [B, maxNB]),
    ``context_lens`` (int32 [B]) and ``free_count`` are updated in place, or the latter
    two into ``out_lens`` and ``out_free_count``; entries past a sequence's length are
    left as they were.  Written too: ``slot_mapping`` and ``positions`` (int64 [T], T at
    least the tokens gained) of the gained tokens, then -1 and 0, and ``cu_seqlens``
    (int32 [B+1]), where each sequence's begin.  Where something does not fit, nothing
    changes and the error flag says what (``include/pa.h`` has the order of blocks, and how
    sequences that share their first blocks begin and end: a block must not be given back
    while another table holds it).
    ``num_blocks`` (default: the capacity) bounds the block ids."""
    rt = _rt or _runtime()
    dev, table = block_tables.get_device(), block_tables.shape
    if out_lens is None:
        out_lens = context_lens
    if out_free_count is None:
        out_free_count = free_count
    if (dev != rt.current_device() or context_lens.get_device() != dev or changes.get_device() != dev or
            free_blocks.get_device() != dev or free_count.get_device() != dev or slot_mapping.get_device() != dev or
            positions.get_device() != dev or cu_seqlens.get_device() != dev or out_lens.get_device() != dev or
            out_free_count.get_device() != dev or not block_tables.is_contiguous() or not context_lens.is_contiguous() or
            not changes.is_contiguous() or not free_blocks.is_contiguous() or not slot_mapping.is_contiguous() or
            not positions.is_contiguous() or not cu_seqlens.is_contiguous() or not out_lens.is_contiguous()):
        _refuse((("block_tables", block_tables), ("context_lens", context_lens), ("changes", changes),
                 ("free_blocks", free_blocks), ("free_count", free_count), ("slot_mapping", slot_mapping),
                 ("positions", positions), ("cu_seqlens", cu_seqlens), ("out_lens", out_lens),
                 ("out_free_count", out_free_count)))
    if len(table) != 2 or block_tables.dtype != rt.i32:
        raise ValueError("block_tables must be int32 [B, maxNB]")
    B = table[0]
    if (context_lens.dtype != rt.i32 or context_lens.numel() != B or changes.dtype != rt.i32 or changes.numel() != B or
            out_lens.dtype != rt.i32 or out_lens.numel() != B):
        raise ValueError("context_lens, changes and out_lens must be int32 [B]")
    if cu_seqlens.dtype != rt.i32 or cu_seqlens.numel() != B + 1:
        raise ValueError("cu_seqlens must be int32 [B+1]")
    if (free_blocks.dtype != rt.i32 or free_count.dtype != rt.i32 or free_count.numel() != 1 or
            out_free_count.dtype != rt.i32 or out_free_count.numel() != 1):
        raise ValueError("free_blocks must be int32 [capacity], free_count and out_free_count int32 [1]")
    if slot_mapping.dtype != rt.i64 or positions.dtype != rt.i64 or positions.numel() != slot_mapping.numel():
        raise ValueError("slot_mapping and positions must be int64 [T]")
    capacity = free_blocks.numel()
    st = rt.lib.pa_update_tables(
        block_tables.data_ptr(), table[1], context_lens.data_ptr(), changes.data_ptr(), out_lens.data_ptr(), B,
        free_blocks.data_ptr(), capacity, free_count.data_ptr(), out_free_count.data_ptr(),
        max(1, capacity) if num_blocks is None else num_blocks, block_size, cu_seqlens.data_ptr(), slot_mapping.data_ptr(),
        positions.data_ptr(), slot_mapping.numel(), None if err_flag is None else _flag(err_flag, dev), rt.stream(dev))
    if st:
        _lib.check(st, "pa_update_tables")


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None, scale: float = 1.0,
                     original_len: int = 4096, fast_turns: float = 32.0, slow_turns: float = 1.0, device=None):
    """(``inv_freq``, ``factor``) for :func:`rope_and_cache`: the angles per position,
    f_i = base^(-2i / rot_dim) (float64 [rot_dim / 2] on the GPU), and the factor on
    turned pairs, for a context ``scale`` times longer than the ``original_len`` positions
    a model was trained on:

    None      f_i as they are
    "linear"  f_i / scale: positions pressed together
    "base"    f_i of the base grown by scale^(rot_dim / (rot_dim - 2)): the slowest pair
              is slowed by scale, the fastest not at all
    "parts"   pairs that turn at least ``fast_turns`` times in original_len positions as
              they are, those that turn at most ``slow_turns`` times slowed by scale, the
              others in between; factor 0.1 ln(scale) + 1

    The ramp of "parts" goes by a pair's turns.  A model whose ramp goes by the pair's index
    between two rounded borders brings an ``inv_freq`` of its own; one that has the ramp
    without the factor passes ``factor=1.0``."""
    torch = _torch()
    _need(rot_dim >= 8 and rot_dim % 8 == 0, "rot_dim must be a multiple of 8")
    _need(base > 1.0 and scale >= 1.0 and math.isfinite(base) and math.isfinite(scale),
          "base must be above 1 and scale at least 1")
    n, factor = rot_dim // 2, 1.0
    if scaling == "base":
        base = base * scale ** (rot_dim / (rot_dim - 2))
    freq = [base ** (-i / n) for i in range(n)]
    if scaling == "linear":
        freq = [f / scale for f in freq]
    elif scaling == "parts":
        _need(fast_turns > slow_turns, "fast_turns must be above slow_turns")
        for i, f in enumerate(freq):
            turns = original_len * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - slow_turns) / (fast_turns - slow_turns)))
            freq[i] = f * keep + f / scale * (1.0 - keep)
        factor = 0.1 * math.log(scale) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError('scaling must be None, "linear", "base" or "parts"')
    return torch.tensor(freq, dtype=torch.float64, device=device or "cuda"), factor


def rope_and_cache(out_q, query, key, value, k_cache, v_cache, slot_mapping, positions, inv_freq, *, interleaved: bool = False,
                   factor: float = 1.0, q_weight=None, k_weight=None, eps: float = 1e-6, k_scales=None, v_scales=None,
                   k_scale: float = 1.0, v_scale: float = 1.0, err_flag=None) -> None:
    """Turn queries [T, Hq, D] into ``out_q`` (which may be ``query``) and keys
    [T, Hkv, D] into the cache, values beside them, in one pass; with ``q_weight`` /
    ``k_weight`` [D] the rows are RMS-normalised per head first.

    Pair i of the first ``2 * inv_freq.numel()`` elements of a row is turned by
    ``positions[t] * inv_freq[i]`` (``inv_freq`` float64 on the GPU, from
    :func:`rope_frequencies`) and multiplied by ``factor``; a pair is the elements
    (i, i + F), or (2i, 2i + 1) if ``interleaved``.  The caches are those of
    :func:`reshape_and_cache` (16-bit, or e4m3 with ``k_scale`` / ``v_scale``), of
    :func:`quant_reshape_and_cache` (with ``k_scales`` / ``v_scales``) or of
    :func:`int4_reshape_and_cache`, told apart by dtype and shape.  query, key and value may be
    slices of one projection's output."""
    rt = _rt or _runtime()
    dev, shape, kshape, cache = query.get_device(), query.shape, key.shape, k_cache.shape
    if (dev != rt.current_device() or out_q.get_device() != dev or key.get_device() != dev or value.get_device() != dev or
            k_cache.get_device() != dev or v_cache.get_device() != dev or slot_mapping.get_device() != dev or
            positions.get_device() != dev or inv_freq.get_device() != dev or not out_q.is_contiguous() or
            not k_cache.is_contiguous() or not v_cache.is_contiguous() or not slot_mapping.is_contiguous() or
            not positions.is_contiguous() or not inv_freq.is_contiguous()):
        _refuse((("out_q", out_q), ("k_cache", k_cache), ("v_cache", v_cache), ("slot_mapping", slot_mapping),
                 ("positions", positions), ("inv_freq", inv_freq)), "query, key and value must be on the device of the caches")
    if len(shape) != 3 or out_q.shape != shape or out_q.dtype != query.dtype:
        raise ValueError("query/out_q must be [T, Hq, D] of one dtype")
    T, hq, d = shape
    if (len(kshape) != 3 or value.shape != kshape or kshape[0] != T or kshape[2] != d or key.dtype != query.dtype or
            value.dtype != query.dtype):
        raise ValueError("key/value must be [T, Hkv, D] of the query's dtype")
    hkv = kshape[1]
    if len(cache) != 4 or v_cache.shape != cache or v_cache.dtype != k_cache.dtype or cache[2] != hkv:
        raise ValueError("caches must be [NB, bs, Hkv, ...] of one dtype, with the rows' heads")
    nb, bs = cache[0], cache[1]
    if (k_scales is None) != (v_scales is None):
        raise ValueError("k_scales and v_scales go together")
    four = k_scales is not None and k_scales.dtype == rt.b16
    if four:
        _int4_cache(rt, k_cache, v_cache, k_scales, v_scales, d)
        code = PA_INT4
    elif cache[3] != d:
        raise ValueError("caches must be [NB, bs, Hkv, D]")
    elif k_scales is not None:
        rows = (nb, bs, hkv)
        if k_scales.shape != rows or v_scales.shape != rows or k_scales.dtype != rt.f32 or v_scales.dtype != rt.f32:
            raise ValueError("scales must be float32 [NB, bs, Hkv] (or bfloat16 for 4-bit codes)")
        code = rt.codes[k_cache.dtype]
    elif k_cache.dtype == query.dtype:
        code = rt.half[k_cache.dtype]
    elif rt.codes.get(k_cache.dtype) == PA_FP8_E4M3:
        code = PA_FP8_E4M3
    else:
        raise TypeError("caches must have the query's dtype, or be e4m3 codes, or come with scales")
    if k_scales is not None and (k_scales.get_device() != dev or v_scales.get_device() != dev or
                                 not k_scales.is_contiguous() or not v_scales.is_contiguous()):
        _refuse((("k_scales", k_scales), ("v_scales", v_scales)))
    if slot_mapping.dtype != rt.i64 or slot_mapping.numel() != T or positions.dtype != rt.i64 or positions.numel() != T:
        raise ValueError("slot_mapping and positions must be int64 [T]")
    if inv_freq.dtype != rt.f64:
        raise ValueError("inv_freq must be float64 [rot_dim / 2]")
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype != query.dtype or w.numel() != d or w.get_device() != dev or not w.is_contiguous()):
            raise ValueError("q_weight/k_weight must be [D] of the query's dtype, on its device")
    qs, ks, vs = query.stride(), key.stride(), value.stride()
    if (qs[2] != 1 or ks[2] != 1 or vs[2] != 1 or (hq != 1 and qs[1] != d) or
            (hkv != 1 and (ks[1] != d or vs[1] != d))):
        raise ValueError("query/key/value: the rows of one token must be dense")
    one = T <= 1
    st = rt.lib.pa_rope_and_cache(
        out_q.data_ptr(), query.data_ptr(), key.data_ptr(), value.data_ptr(), hq * d if one else qs[0],
        hkv * d if one else ks[0], hkv * d if one else vs[0], k_cache.data_ptr(), v_cache.data_ptr(), code,
        None if k_scales is None else k_scales.data_ptr(), None if v_scales is None else v_scales.data_ptr(), k_scale,
        v_scale, slot_mapping.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(), 2 * inv_freq.numel(), interleaved,
        factor, None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(), eps,
        T, hq, hkv, d, rt.half[query.dtype], nb, bs, None if err_flag is None else _flag(err_flag, dev), rt.stream(dev))
    if st:
        _lib.check(st, "pa_rope_and_cache")


@functools.lru_cache(maxsize=1024)
def decode_shared_workspace_size(num_seqs, num_groups, max_group_size, num_heads, num_kv_heads, head_dim, block_size,
                                 max_context_len, max_shared_len, partition_size=0) -> int:
    n = _lib.load().pa_decode_shared_workspace_size(num_seqs, num_groups, max_group_size, num_heads, num_kv_heads,
                                                    head_dim, block_size, max_context_len, max_shared_len,
                                                    partition_size)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("arguments rejected by pa_decode_shared_workspace_size")
    return n


def decode_shared(out, query, k_cache, v_cache, block_tables, context_lens, cu_groups, shared_lens, scale: float,
                  max_group_size: int | None = None, max_shared_len: int | None = None,
                  max_context_len: int | None = None, partition_size: int = 0, workspace=None, err_flag=None) -> None:
    """:func:`decode` for a batch whose sequences share prefixes, each computed
    once for all sequences of its group.

    Group g is the sequences ``cu_groups[g] .. cu_groups[g+1]-1`` (int32 [NG+1]);
    the first ``shared_lens[s]`` tokens (int32 [B], one value per group) hold the
    same K/V rows in every member.  ``max_group_size`` and ``max_shared_len`` are
    host-side bounds (defaults: the batch size and ``max_context_len``; tight
    bounds make the call faster and its workspace smaller:
    :func:`decode_shared_workspace_size`).  A list of groups may be padded with
    empty ones up to any length, as a captured step's is."""
    rt = _rt or _runtime()
    dev, cache = query.get_device(), k_cache.shape
    if (dev != rt.current_device() or out.get_device() != dev or k_cache.get_device() != dev or
            v_cache.get_device() != dev or block_tables.get_device() != dev or context_lens.get_device() != dev or
            cu_groups.get_device() != dev or shared_lens.get_device() != dev or not query.is_contiguous() or
            not out.is_contiguous() or not k_cache.is_contiguous() or not v_cache.is_contiguous() or
            not block_tables.is_contiguous() or not context_lens.is_contiguous() or not cu_groups.is_contiguous() or
            not shared_lens.is_contiguous()):
        _refuse((("query", query), ("out", out), ("k_cache", k_cache), ("v_cache", v_cache),
                 ("block_tables", block_tables), ("context_lens", context_lens), ("cu_groups", cu_groups),
                 ("shared_lens", shared_lens)))
    _decode_shapes(rt, out, query, cache, v_cache, block_tables, context_lens)
    if k_cache.dtype != query.dtype or v_cache.dtype != query.dtype:
        raise ValueError("caches must have the query's dtype")
    B, Hq, D = query.shape
    nb, bs, hkv, _ = cache
    ng = cu_groups.numel() - 1
    if cu_groups.dtype != rt.i32 or cu_groups.dim() != 1 or ng < 0:
        raise ValueError("cu_groups must be int32 [NG+1]")
    if shared_lens.dtype != rt.i32 or shared_lens.numel() != B:
        raise ValueError("shared_lens must be int32 [B]")
    maxnb = block_tables.shape[1]
    if max_context_len is None:
        max_context_len = maxnb * bs
    if max_group_size is None:
        max_group_size = B
    if max_shared_len is None:
        max_shared_len = max_context_len
    stream = rt.stream(dev)
    buf = _scratch(rt, workspace, decode_shared_workspace_size(B, ng, max_group_size, Hq, hkv, D, bs, max_context_len,
                                                               max_shared_len, partition_size), dev, stream)
    st = rt.lib.pa_decode_shared(
        out.data_ptr(), rt.out[out.dtype], query.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        rt.half[query.dtype], block_tables.data_ptr(), maxnb, context_lens.data_ptr(), max_context_len,
        cu_groups.data_ptr(), ng, max_group_size, shared_lens.data_ptr(), max_shared_len, B, Hq, hkv, D, bs, nb, scale,
        partition_size, None if buf is None else buf.data_ptr(), 0 if buf is None else buf.nbytes,
        None if err_flag is None else _flag(err_flag, dev), stream)
    if st:
        _lib.check(st, "pa_decode_shared")


class StepGraph:
    """A step of this library's calls captured once as a CUDA graph and then
    replayed with one launch, as a serving loop does for its decode step.

    ``fn()`` enqueues the step (e.g. :func:`reshape_and_cache` then
    :func:`decode`) on the current stream, on device buffers that stay
    allocated at the same addresses for the graph's lifetime; refill those
    buffers in place between replays.  Everything ``fn`` needs is allocated
    before capture: it is run ``warmup`` times first (so default workspaces
    exist), and workspaces passed to it must already be large enough.  The
    argument checks of each call run at capture; a replay launches the
    captured kernels (with their programmatic dependent launch edges) as they
    were.
    """

    def __init__(self, fn, warmup: int = 1):
        torch = _torch()
        self._fn = fn
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(max(1, warmup)):
                fn()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            fn()
        torch.cuda.synchronize()

    def replay(self) -> None:
        """Launch the captured step on the current stream."""
        self.graph.replay()
