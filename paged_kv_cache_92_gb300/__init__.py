"""Python binding of libpagedkv.so: paged KV-cache decode attention on GB300.

Argument marshalling only. Every step of the data path runs in the CUDA
kernels of ``libpagedkv.so`` (see ``include/pagedkv.h``); torch supplies
device memory and streams. There is no CPU fallback: if the library has not
been built, every call raises. Calls run on the current CUDA device, and refuse
(``ValueError``) tensors that are not on it.

Names follow the C ABI: ``pa_decode``, ``pa_decode_workspace_size``,
``pa_reshape_and_cache``, ``pa_copy_blocks``, ``pa_device_errors`` and the
``pa_pool_*`` / ``pa_seq_*`` block-pool calls (wrapped by ``Pool``). The cache
calls have forms for the 8-bit (``_fp8``) and the 4-bit (``_fp4``) cache;
``pa_token_weights``, ``pa_evict_select``, ``pa_evict_compact`` and
``Pool.compact`` evict tokens; ``pa_update_tables`` keeps tables on the device;
``pa_block_bounds``, ``pa_block_scores``, ``pa_block_select`` and
``pa_decode_selected`` attend to the blocks that matter.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import List, Optional, Sequence, Tuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpagedkv.so")

PA_OK = 0
STATUS_NAMES = {0: "PA_OK", 1: "PA_ERR_INVALID_ARG", 2: "PA_ERR_UNSUPPORTED", 3: "PA_ERR_OOM",
                4: "PA_ERR_REFCOUNT", 5: "PA_ERR_BOUNDS", 6: "PA_ERR_CUDA"}
DEVERR_TABLE_ENTRY = 0x1
DEVERR_CONTEXT_LEN = 0x2
DEVERR_SLOT = 0x4
DEVERR_COPY_PAIR = 0x8
DEVERR_TIMEOUT = 0x10
DEVERR_APPEND_SLOT = 0x20
DEVERR_KEEP = 0x40
DEVERR_POOL = 0x80

KV_BF16 = 0
KV_FP8_E4M3 = 1
KV_FP4_E2M1 = 2

EXPORTED_SYMBOLS = [
    "pa_status_string", "pa_last_error", "pa_version", "pa_device_errors",
    "pa_decode_workspace_size", "pa_decode", "pa_decode_noalloc", "pa_append_decode",
    "pa_step_host_layout", "pa_step_host_workspace_size", "pa_step_host",
    "pa_reshape_and_cache", "pa_reshape_and_cache_fp8", "pa_copy_blocks_fp8",
    "pa_reshape_and_cache_fp4", "pa_gather_fp4", "pa_copy_blocks_fp4",
    "pa_copy_blocks",
    "pa_token_weights_workspace_size", "pa_token_weights", "pa_evict_select",
    "pa_evict_compact", "pa_pool_compact",
    "pa_update_tables", "pa_block_bounds", "pa_block_scores", "pa_block_select",
    "pa_decode_selected_workspace_size", "pa_decode_selected",
    "pa_pool_create", "pa_pool_destroy", "pa_pool_alloc", "pa_pool_incref", "pa_pool_decref",
    "pa_pool_refcount", "pa_pool_stats", "pa_seq_create", "pa_seq_free", "pa_seq_fork",
    "pa_seq_append_slot", "pa_seq_append_tokens", "pa_seq_length", "pa_seq_table",
    "pa_pool_export", "pa_seq_create_prompt", "pa_pool_prefix_stats",
]


class PagedKVError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {detail}")


class PoolOOM(PagedKVError):
    pass


class DecodeParams(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("block_tables", ctypes.c_void_p), ("context_lens", ctypes.c_void_p),
        ("max_blocks_per_seq", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32), ("max_context_len", ctypes.c_int32),
        ("scale", ctypes.c_float), ("partition_tokens", ctypes.c_int32),
        ("variant", ctypes.c_int32), ("overlap_prologue", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("query_len", ctypes.c_int32), ("wait_timeout_us", ctypes.c_int32),
    ]


DECODE_TENSOR_CORE = 0
DECODE_CUDA_CORE = 1


class AppendParams(ctypes.Structure):
    _fields_ = [
        ("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
        ("slot_mapping", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
    ]


class TokenWeightsParams(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p),
        ("block_tables", ctypes.c_void_p), ("context_lens", ctypes.c_void_p),
        ("token_weights", ctypes.c_void_p), ("weights_stride", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32), ("max_context_len", ctypes.c_int32),
        ("scale", ctypes.c_float), ("kv_dtype", ctypes.c_int32), ("k_scale", ctypes.c_void_p),
        ("query_len", ctypes.c_int32), ("accumulate", ctypes.c_int32),
    ]


class EvictCompactParams(ctypes.Structure):
    _fields_ = [
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("block_tables", ctypes.c_void_p), ("dst_tables", ctypes.c_void_p),
        ("keep", ctypes.c_void_p), ("new_lens", ctypes.c_void_p),
        ("token_weights", ctypes.c_void_p), ("weights_stride", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32), ("max_dst_blocks_per_seq", ctypes.c_int32),
        ("keep_stride", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
    ]


class UpdateTablesParams(ctypes.Structure):
    _fields_ = [
        ("block_tables", ctypes.c_void_p), ("old_lens", ctypes.c_void_p),
        ("new_lens", ctypes.c_void_p), ("free_ring", ctypes.c_void_p),
        ("ring_state", ctypes.c_void_p), ("new_ring_state", ctypes.c_void_p),
        ("slot_mapping", ctypes.c_void_p), ("positions", ctypes.c_void_p),
        ("token_starts", ctypes.c_void_p),
        ("max_blocks_per_seq", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
        ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
        ("ring_size", ctypes.c_int32), ("max_new_tokens", ctypes.c_int32),
    ]


class BlockBoundsParams(ctypes.Structure):
    _fields_ = [
        ("k_cache", ctypes.c_void_p), ("bounds", ctypes.c_void_p),
        ("block_tables", ctypes.c_void_p), ("context_lens", ctypes.c_void_p),
        ("old_lens", ctypes.c_void_p),
        ("max_blocks_per_seq", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
        ("max_new_tokens", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
    ]


class BlockScoresParams(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("bounds", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
        ("block_tables", ctypes.c_void_p), ("context_lens", ctypes.c_void_p),
        ("scores", ctypes.c_void_p), ("scores_stride", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32), ("max_context_len", ctypes.c_int32),
        ("scale", ctypes.c_float), ("query_len", ctypes.c_int32),
    ]


class StepLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in
                ("q", "k_new", "v_new", "slot_mapping", "block_tables", "context_lens",
                 "cow_pairs", "total")]


class StepHostParams(ctypes.Structure):
    _fields_ = [
        ("host_in", ctypes.c_void_p), ("host_out", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("num_seqs", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32), ("max_context_len", ctypes.c_int32),
        ("num_cow_pairs", ctypes.c_int32), ("scale", ctypes.c_float), ("variant", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("query_len", ctypes.c_int32),
    ]


class PrefixStats(ctypes.Structure):
    _fields_ = [("cached_blocks", ctypes.c_int32), ("evictable_blocks", ctypes.c_int32),
                ("lookups", ctypes.c_int64), ("hits", ctypes.c_int64)]


class PoolStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("num_blocks", "block_size", "free_blocks", "used_blocks", "shared_blocks",
                 "max_refcount", "live_seqs")]


_lib = None


def load():
    """Load libpagedkv.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: run paged_kv_cache_92_gb300.build.build() "
                          "(or __graft_entry__.build()) first; there is no fallback path")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    P = ctypes.POINTER
    sigs = {
        "pa_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "pa_last_error": ([], ctypes.c_char_p),
        "pa_version": ([], i32),
        "pa_device_errors": ([vp, P(ctypes.c_uint32)], ctypes.c_int),
        "pa_decode_workspace_size": ([P(DecodeParams)], sz),
        "pa_decode": ([P(DecodeParams), vp, sz, vp], ctypes.c_int),
        "pa_decode_noalloc": ([P(DecodeParams), vp], ctypes.c_int),
        "pa_append_decode": ([P(DecodeParams), P(AppendParams), vp, sz, vp], ctypes.c_int),
        "pa_step_host_layout": ([P(StepHostParams), P(StepLayout)], ctypes.c_int),
        "pa_step_host_workspace_size": ([P(StepHostParams)], sz),
        "pa_step_host": ([P(StepHostParams), vp, sz, vp], ctypes.c_int),
        "pa_reshape_and_cache": ([vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp], ctypes.c_int),
        "pa_copy_blocks": ([vp, vp, vp, i32, i32, i32, i32, i32, vp], ctypes.c_int),
        "pa_reshape_and_cache_fp8": ([vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp],
                                     ctypes.c_int),
        "pa_copy_blocks_fp8": ([vp, vp, vp, i32, i32, i32, i32, i32, vp], ctypes.c_int),
        "pa_reshape_and_cache_fp4": ([vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp],
                                     ctypes.c_int),
        "pa_gather_fp4": ([vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp], ctypes.c_int),
        "pa_copy_blocks_fp4": ([vp, vp, vp, i32, i32, i32, i32, i32, vp], ctypes.c_int),
        "pa_token_weights_workspace_size": ([P(TokenWeightsParams)], sz),
        "pa_token_weights": ([P(TokenWeightsParams), vp, sz, vp], ctypes.c_int),
        "pa_evict_select": ([vp, vp, vp, vp, i32, i32, i32, i32, vp], ctypes.c_int),
        "pa_evict_compact": ([P(EvictCompactParams), vp], ctypes.c_int),
        "pa_pool_compact": ([vp, vp, vp, i32], ctypes.c_int),
        "pa_update_tables": ([P(UpdateTablesParams), vp], ctypes.c_int),
        "pa_block_bounds": ([P(BlockBoundsParams), vp], ctypes.c_int),
        "pa_block_scores": ([P(BlockScoresParams), vp], ctypes.c_int),
        "pa_block_select": ([vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp], ctypes.c_int),
        "pa_decode_selected_workspace_size": ([P(DecodeParams), i32], sz),
        "pa_decode_selected": ([P(DecodeParams), vp, i32, vp, sz, vp], ctypes.c_int),
        "pa_pool_create": ([i32, i32, vp, P(vp)], ctypes.c_int),
        "pa_pool_destroy": ([vp], None),
        "pa_pool_alloc": ([vp, P(i32)], ctypes.c_int),
        "pa_pool_incref": ([vp, i32], ctypes.c_int),
        "pa_pool_decref": ([vp, i32], ctypes.c_int),
        "pa_pool_refcount": ([vp, i32], i32),
        "pa_pool_stats": ([vp, P(PoolStats)], ctypes.c_int),
        "pa_seq_create": ([vp, P(i32)], ctypes.c_int),
        "pa_seq_free": ([vp, i32], ctypes.c_int),
        "pa_seq_fork": ([vp, i32, i32, P(i32)], ctypes.c_int),
        "pa_seq_append_slot": ([vp, i32, P(i64), P(i32), P(i32)], ctypes.c_int),
        "pa_seq_append_tokens": ([vp, i32, i32, vp, vp, P(i32)], ctypes.c_int),
        "pa_seq_length": ([vp, i32, P(i32)], ctypes.c_int),
        "pa_seq_table": ([vp, i32, vp, i32, P(i32)], ctypes.c_int),
        "pa_pool_export": ([vp, vp, i32, i32, vp, vp], ctypes.c_int),
        "pa_seq_create_prompt": ([vp, vp, i32, P(i32), P(i32), vp], ctypes.c_int),
        "pa_pool_prefix_stats": ([vp, P(PrefixStats)], ctypes.c_int),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(status: int, where: str) -> None:
    if status != PA_OK:
        detail = load().pa_last_error().decode(errors="replace")
        cls = PoolOOM if status == 3 else PagedKVError
        raise cls(status, where, detail)


# --------------------------------------------------------------------------
# device calls (torch tensors in, marshalled to raw pointers)
# --------------------------------------------------------------------------

# torch's calls for the current device, looked up once: the checks below run for
# every tensor of every call, and a step is a few microseconds
_device = _raw_stream = None
_i32 = _i64 = _f32 = _bf16 = _u8 = None


def _bind_torch() -> None:
    global _device, _raw_stream, _i32, _i64, _f32, _bf16, _u8
    import torch

    _i32, _i64, _f32 = torch.int32, torch.int64, torch.float32
    _bf16, _u8 = torch.bfloat16, torch.uint8
    _raw_stream = torch._C._cuda_getCurrentRawStream
    _device = torch._C._cuda_getDevice


def _current() -> Optional[int]:
    """The current device, for ``_ptr``; None where there is none (every tensor is then
    refused by ``_dev_ptr``). Binds torch."""
    if _device is None:
        _bind_torch()
    try:
        return _device()
    except Exception:
        return None


def _ptr(t, dtype, name: str, device: Optional[int]) -> int:
    """``_dev_ptr`` for a call of many tensors: the current device is looked up once."""
    try:
        if t.dtype is dtype and t.is_contiguous() and t.is_cuda and t.get_device() == device:
            return t.data_ptr()
    except AttributeError:
        pass
    return _dev_ptr(t, dtype, name)


def _dev_ptr(t, dtype, name: str) -> int:
    if _device is None:
        _bind_torch()
    try:  # one condition for the tensor that passes (without a driver _device() raises)
        if t.dtype is dtype and t.is_contiguous() and t.is_cuda and t.get_device() == _device():
            return t.data_ptr()
    except AttributeError:
        pass
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must live on the current CUDA device")


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        if _device is None:
            _bind_torch()
        # the handle alone: a Stream object costs a call several microseconds
        return _raw_stream(_device()) or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _empty(stream, like, shape, dtype):
    """Uninitialised memory for a call on ``stream``, from that stream's pool of the
    caching allocator: what lies there then neither waits for other streams' work
    nor, once dropped, is handed to them while the call still runs."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def kv_cache_format(k_cache) -> Tuple[int, int]:
    """(kv_dtype, head_dim) of a K cache tensor: bf16 [NB][Hkv][BS][D]; uint8
    [NB][Hkv][BS][D] for the 8-bit cache, [NB][Hkv][BS][D * 9 / 16] for the
    4-bit one (36 or 72 bytes a row: no 8-bit head_dim)."""
    if _u8 is None:
        _bind_torch()
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError("a cache is [num_blocks][num_kv_heads][block_size][row]")
    row = shape[3]
    if k_cache.dtype is _u8:
        return (KV_FP4_E2M1, row * 16 // 9) if row in (36, 72) else (KV_FP8_E4M3, row)
    return KV_BF16, row


def fp4_cache_shape(num_blocks: int, num_kv_heads: int, block_size: int, head_dim: int):
    """Shape of a 4-bit K or V cache (uint8). The last two dimensions are one
    tile's bytes (codes of all its rows, then their scales), not its rows."""
    if head_dim not in (64, 128):
        raise ValueError("the 4-bit cache takes head_dim 64 or 128")
    return (num_blocks, num_kv_heads, block_size, head_dim * 9 // 16)


def _v_cache_ok(fmt: int, k_cache, v_cache) -> bool:
    if fmt == KV_FP8_E4M3:
        return tuple(v_cache.shape) in fp8_v_shapes(*k_cache.shape)
    return v_cache.shape == k_cache.shape


def make_decode_params(q, out, k_cache, v_cache, block_tables, context_lens,
                       max_context_len: int, scale: Optional[float] = None,
                       partition_tokens: int = 0, variant: int = DECODE_TENSOR_CORE,
                       overlap_prologue: bool = False, k_scale=None,
                       v_scale=None, wait_timeout_us: int = 0) -> DecodeParams:
    """Marshal a pa_decode call. q and out are bf16 [B][Hq][D] (one new token
    per sequence) or [B][Q][Hq][D] (Q new tokens per sequence, causal among
    them). bf16 caches [NB][Hkv][BS][D]; uint8 caches are the 8-bit E4M3 cache
    (K [NB][Hkv][BS][D], V^T in 16-key sub-tiles [NB][Hkv][BS/16][D][16]) or,
    with D * 9 / 16 bytes a row, the 4-bit cache (``fp4_cache_shape``); both
    need k_scale / v_scale, float32 CUDA tensors [Hkv]."""
    dev = _current()
    shape = q.shape
    if len(shape) == 4:
        B, QL, Hq, D = shape
    else:
        (B, Hq, D), QL = shape, 0
    fmt, D2 = kv_cache_format(k_cache)
    NB, Hkv, BS, _ = k_cache.shape
    if D2 != D or not _v_cache_ok(fmt, k_cache, v_cache) or out.shape != shape:
        raise ValueError("shape mismatch between q / out / k_cache / v_cache")
    tables = block_tables.shape
    if len(tables) != 2 or tables[0] != B or context_lens.shape != (B,):
        raise ValueError("block_tables must be [num_seqs][max_blocks], context_lens [num_seqs]")
    fmt_dtype = _bf16 if fmt == KV_BF16 else _u8
    ks = vs = None
    if fmt != KV_BF16:
        if k_scale is None or v_scale is None:
            raise ValueError("the 8-bit and 4-bit caches need k_scale and v_scale")
        ks = _ptr(k_scale, _f32, "k_scale", dev)
        vs = _ptr(v_scale, _f32, "v_scale", dev)
        if fmt == KV_FP4_E2M1 and (k_scale.numel() != Hkv or v_scale.numel() != Hkv):
            raise ValueError("k_scale and v_scale must be [num_kv_heads]")
    return DecodeParams(
        _ptr(q, _bf16, "q", dev), _ptr(out, _bf16, "out", dev),
        _ptr(k_cache, fmt_dtype, "k_cache", dev), _ptr(v_cache, fmt_dtype, "v_cache", dev),
        _ptr(block_tables, _i32, "block_tables", dev),
        _ptr(context_lens, _i32, "context_lens", dev),
        tables[1], B, Hq, Hkv, D, BS, NB, int(max_context_len),
        float(1.0 / math.sqrt(D) if scale is None else scale), int(partition_tokens),
        int(variant), int(bool(overlap_prologue)), fmt, ks, vs, int(QL), int(wait_timeout_us))


def pa_decode_workspace_size(params: DecodeParams) -> int:
    return int(load().pa_decode_workspace_size(ctypes.byref(params)))


def pa_decode(q, k_cache, v_cache, block_tables, context_lens, max_context_len: int,
              scale: Optional[float] = None, partition_tokens: int = 0, out=None,
              workspace=None, stream=None, variant: int = DECODE_TENSOR_CORE,
              overlap_prologue: bool = False, k_scale=None, v_scale=None,
              wait_timeout_us: int = 0):
    """Paged decode attention; returns ``out`` (bf16, the shape of ``q``:
    [B][Hq][d], or [B][Q][Hq][d] for Q new tokens per sequence).

    ``workspace`` is a uint8 CUDA tensor of at least
    ``pa_decode_workspace_size`` bytes; allocated here when omitted.
    """
    import torch

    lib = load()
    if out is None:
        out = _empty(stream, q, q.shape, q.dtype)
    p = make_decode_params(q, out, k_cache, v_cache, block_tables, context_lens,
                           max_context_len, scale, partition_tokens, variant, overlap_prologue,
                           k_scale, v_scale, wait_timeout_us)
    if workspace is None:
        need = int(lib.pa_decode_workspace_size(ctypes.byref(p)))
        if need > 0:
            workspace = _empty(stream, q, need, torch.uint8)
    ws_ptr = _dev_ptr(workspace, torch.uint8, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check(lib.pa_decode(ctypes.byref(p), ws_ptr, ws_bytes, _stream_handle(stream)), "pa_decode")
    return out


def make_append_params(k_new, v_new, slot_mapping, k_cache, v_cache) -> AppendParams:
    import torch

    T, Hkv, D = k_new.shape  # T = num_seqs * (new tokens per sequence)
    if tuple(v_new.shape) != (T, Hkv, D) or tuple(slot_mapping.shape) != (T,) \
            or tuple(k_cache.shape[1:2]) != (Hkv,) or kv_cache_format(k_cache)[1] != D:
        raise ValueError("k_new/v_new must be [num_seqs * Q][num_kv_heads][head_dim] matching "
                         "the cache, slot_mapping [num_seqs * Q]")
    a = AppendParams()
    a.k_new = _dev_ptr(k_new, torch.bfloat16, "k_new")
    a.v_new = _dev_ptr(v_new, torch.bfloat16, "v_new")
    a.slot_mapping = _dev_ptr(slot_mapping, torch.int64, "slot_mapping")
    cache_dtype = torch.uint8 if k_cache.dtype == torch.uint8 else torch.bfloat16
    a.k_cache = _dev_ptr(k_cache, cache_dtype, "k_cache")
    a.v_cache = _dev_ptr(v_cache, cache_dtype, "v_cache")
    return a


def pa_append_decode(q, k_cache, v_cache, block_tables, context_lens, max_context_len: int,
                     k_new, v_new, slot_mapping, scale: Optional[float] = None,
                     partition_tokens: int = 0, out=None, workspace=None, stream=None,
                     variant: int = DECODE_TENSOR_CORE, overlap_prologue: bool = False,
                     k_scale=None, v_scale=None):
    """One decode step in one launch: write token b's K/V (``k_new[b]``,
    ``v_new[b]``) at ``slot_mapping[b]`` -- which must be the slot of token
    ``context_lens[b] - 1`` of sequence b -- then paged decode attention over
    the updated caches. Same result as ``pa_reshape_and_cache`` followed by
    ``pa_decode``; returns ``out``. With q [B][Q][Hq][d], row b*Q + i of
    ``k_new``/``v_new``/``slot_mapping`` is token ``context_lens[b] - Q + i``.
    For the 8-bit cache (uint8 caches, with ``k_scale``/``v_scale``) the write
    is the quantising one of ``pa_reshape_and_cache_fp8``, for the 4-bit cache
    that of ``pa_reshape_and_cache_fp4``."""
    import torch

    lib = load()
    if out is None:
        out = _empty(stream, q, q.shape, q.dtype)
    p = make_decode_params(q, out, k_cache, v_cache, block_tables, context_lens,
                           max_context_len, scale, partition_tokens, variant, overlap_prologue,
                           k_scale, v_scale)
    a = make_append_params(k_new, v_new, slot_mapping, k_cache, v_cache)
    need = int(lib.pa_decode_workspace_size(ctypes.byref(p)))
    if workspace is None and need > 0:
        workspace = _empty(stream, q, need, torch.uint8)
    ws_ptr = _dev_ptr(workspace, torch.uint8, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check(lib.pa_append_decode(ctypes.byref(p), ctypes.byref(a), ws_ptr, ws_bytes,
                                _stream_handle(stream)), "pa_append_decode")
    return out


def make_step_host_params(k_cache, v_cache, num_seqs: int, num_q_heads: int,
                          max_blocks_per_seq: int, max_context_len: int, num_cow_pairs: int = 0,
                          scale: Optional[float] = None,
                          variant: int = DECODE_TENSOR_CORE, k_scale=None,
                          v_scale=None, query_len: int = 0) -> StepHostParams:
    """Shape half of a host-driven step; host_in / host_out are set by the caller
    (or by ``pa_step_host``). uint8 caches are the 8-bit (E4M3) or 4-bit cache and
    need ``k_scale`` / ``v_scale`` (float32 CUDA tensors [num_kv_heads]). With
    ``query_len`` Q > 1 every sequence brings Q new tokens (the layouts of
    ``pa_append_decode``)."""
    import torch

    NB, Hkv, BS, _ = k_cache.shape
    p = StepHostParams()
    fmt, D = kv_cache_format(k_cache)
    cache_dtype = torch.bfloat16 if fmt == KV_BF16 else torch.uint8
    p.k_cache = _dev_ptr(k_cache, cache_dtype, "k_cache")
    p.v_cache = _dev_ptr(v_cache, cache_dtype, "v_cache")
    if fmt == KV_FP4_E2M1 and not _v_cache_ok(fmt, k_cache, v_cache):
        raise ValueError("shape mismatch between k_cache and v_cache")
    if fmt != KV_BF16:
        if k_scale is None or v_scale is None:
            raise ValueError("the 8-bit and 4-bit caches need k_scale and v_scale")
        if fmt == KV_FP4_E2M1 and (k_scale.numel() != Hkv or v_scale.numel() != Hkv):
            raise ValueError("k_scale and v_scale must be [num_kv_heads]")
        p.kv_dtype = fmt
        p.k_scale = _dev_ptr(k_scale, torch.float32, "k_scale")
        p.v_scale = _dev_ptr(v_scale, torch.float32, "v_scale")
    p.num_seqs, p.num_q_heads, p.num_kv_heads, p.head_dim = num_seqs, num_q_heads, Hkv, D
    p.block_size, p.num_blocks = BS, NB
    p.max_blocks_per_seq, p.max_context_len = max_blocks_per_seq, int(max_context_len)
    p.num_cow_pairs = num_cow_pairs
    p.scale = float(1.0 / math.sqrt(D) if scale is None else scale)
    p.variant = int(variant)
    p.query_len = int(query_len)
    return p


def pa_step_host_layout(params: StepHostParams) -> StepLayout:
    out = StepLayout()
    _check(load().pa_step_host_layout(ctypes.byref(params), ctypes.byref(out)),
           "pa_step_host_layout")
    return out


def pa_step_host_workspace_size(params: StepHostParams) -> int:
    return int(load().pa_step_host_workspace_size(ctypes.byref(params)))


def pack_step_inputs(params: StepHostParams, q, k_new, v_new, slot_mapping, block_tables,
                     context_lens, cow_pairs=None, pin: bool = True):
    """Marshal one step's host inputs into the packed buffer of ``pa_step_host``
    (a uint8 CPU tensor; pinned unless ``pin`` is False)."""
    import torch

    L = pa_step_host_layout(params)
    buf = torch.zeros(int(L.total), dtype=torch.uint8, pin_memory=pin)
    parts = [(L.q, q, torch.bfloat16), (L.k_new, k_new, torch.bfloat16),
             (L.v_new, v_new, torch.bfloat16), (L.slot_mapping, slot_mapping, torch.int64),
             (L.block_tables, block_tables, torch.int32), (L.context_lens, context_lens, torch.int32)]
    if params.num_cow_pairs:
        parts.append((L.cow_pairs, cow_pairs, torch.int32))
    for off, t, dt in parts:
        t = torch.as_tensor(t).to("cpu", dt).contiguous().view(torch.uint8).reshape(-1)
        buf[int(off):int(off) + t.numel()] = t
    return buf


def pa_step_host(params: StepHostParams, host_in, host_out, workspace, stream=None) -> None:
    """One whole step from host memory (see the C header): ``host_in`` is a
    uint8 CPU tensor packed by ``pa_step_host_layout`` (pinned for speed),
    ``host_out`` a bf16 CPU tensor [num_seqs][num_q_heads][head_dim] (with Q new
    tokens per sequence [num_seqs][Q][num_q_heads][head_dim]),
    ``workspace`` a uint8 CUDA tensor. Returns when host_out holds the result."""
    import torch

    if host_in.device.type != "cpu" or host_out.device.type != "cpu":
        raise ValueError("host_in and host_out must be host (CPU) tensors")
    if not host_in.is_contiguous() or not host_out.is_contiguous():
        raise ValueError("host_in and host_out must be contiguous")
    if host_out.dtype != torch.bfloat16 or host_in.dtype != torch.uint8:
        raise ValueError("host_in must be uint8, host_out bf16")
    params.host_in = host_in.data_ptr()
    params.host_out = host_out.data_ptr()
    ws = _dev_ptr(workspace, torch.uint8, "workspace")
    _check(load().pa_step_host(ctypes.byref(params), ws, workspace.numel(),
                               _stream_handle(stream)), "pa_step_host")


def pa_decode_noalloc(q, k_cache, v_cache, block_tables, context_lens, max_context_len: int,
                      scale: Optional[float] = None, partition_tokens: int = 0, out=None,
                      stream=None, variant: int = DECODE_TENSOR_CORE, k_scale=None, v_scale=None):
    """Same decode as ``pa_decode`` without any workspace: for callers that
    cannot allocate device memory at decode time (all free HBM already handed
    to the KV pool, or no room for cudaMalloc's synchronisation in the serving
    loop). The split-K partials live in a fixed 16 MiB device array inside the
    library; larger needs are rejected. ``out`` must be given by such callers;
    when omitted it is allocated here for convenience. Calls that overlap on
    the GPU share that array and race."""
    lib = load()
    if out is None:
        out = _empty(stream, q, q.shape, q.dtype)
    p = make_decode_params(q, out, k_cache, v_cache, block_tables, context_lens,
                           max_context_len, scale, partition_tokens, variant, k_scale=k_scale,
                           v_scale=v_scale)
    _check(lib.pa_decode_noalloc(ctypes.byref(p), _stream_handle(stream)), "pa_decode_noalloc")
    return out


def pa_reshape_and_cache(k_new, v_new, k_cache, v_cache, slot_mapping, stream=None) -> None:
    import torch

    T, Hkv, D = k_new.shape
    NB, Hkv2, BS, D2 = k_cache.shape
    if (Hkv2, D2) != (Hkv, D) or tuple(v_new.shape) != tuple(k_new.shape) \
            or tuple(v_cache.shape) != tuple(k_cache.shape) or tuple(slot_mapping.shape) != (T,):
        raise ValueError("shape mismatch in pa_reshape_and_cache")
    lib = load()
    _check(lib.pa_reshape_and_cache(
        _dev_ptr(k_new, torch.bfloat16, "k_new"), _dev_ptr(v_new, torch.bfloat16, "v_new"),
        _dev_ptr(k_cache, torch.bfloat16, "k_cache"), _dev_ptr(v_cache, torch.bfloat16, "v_cache"),
        _dev_ptr(slot_mapping, torch.int64, "slot_mapping"), T, Hkv, D, BS, NB,
        _stream_handle(stream)), "pa_reshape_and_cache")


def pa_copy_blocks(k_cache, v_cache, pairs, stream=None) -> None:
    import torch

    NB, Hkv, BS, D = k_cache.shape
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be int32 [n][2]")
    lib = load()
    _check(lib.pa_copy_blocks(
        _dev_ptr(k_cache, torch.bfloat16, "k_cache"), _dev_ptr(v_cache, torch.bfloat16, "v_cache"),
        _dev_ptr(pairs, torch.int32, "pairs"), pairs.shape[0], Hkv, D, BS, NB,
        _stream_handle(stream)), "pa_copy_blocks")


def fp8_v_shapes(NB: int, Hkv: int, BS: int, D: int):
    """Shapes accepted for the 8-bit V^T cache: [NB][Hkv][BS/W][D][W] (sub-tiles
    of W = min(BS, 16) keys), and up to block size 16 also [NB][Hkv][D][W]."""
    W = min(BS, 16)
    shapes = [(NB, Hkv, BS // W, D, W)]
    if BS <= 16:
        shapes.append((NB, Hkv, D, W))
    return shapes


def pa_reshape_and_cache_fp8(k_new, v_new, k_cache, v_cache, slot_mapping, k_scale, v_scale,
                             stream=None) -> None:
    """KV write into the 8-bit cache (uint8 K [NB][Hkv][BS][D], V^T in sub-tiles
    of W = min(BS, 16) keys, [NB][Hkv][BS/W][D][W])."""
    import torch

    T, Hkv, D = k_new.shape
    NB, Hkv2, BS, D2 = k_cache.shape
    if (Hkv2, D2) != (Hkv, D) or tuple(v_new.shape) != tuple(k_new.shape) \
            or tuple(v_cache.shape) not in fp8_v_shapes(NB, Hkv, BS, D) \
            or tuple(slot_mapping.shape) != (T,):
        raise ValueError("shape mismatch in pa_reshape_and_cache_fp8")
    lib = load()
    _check(lib.pa_reshape_and_cache_fp8(
        _dev_ptr(k_new, torch.bfloat16, "k_new"), _dev_ptr(v_new, torch.bfloat16, "v_new"),
        _dev_ptr(k_cache, torch.uint8, "k_cache"), _dev_ptr(v_cache, torch.uint8, "v_cache"),
        _dev_ptr(slot_mapping, torch.int64, "slot_mapping"),
        _dev_ptr(k_scale, torch.float32, "k_scale"), _dev_ptr(v_scale, torch.float32, "v_scale"),
        T, Hkv, D, BS, NB, _stream_handle(stream)), "pa_reshape_and_cache_fp8")


def pa_copy_blocks_fp8(k_cache, v_cache, pairs, stream=None) -> None:
    import torch

    NB, Hkv, BS, D = k_cache.shape
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be int32 [n][2]")
    lib = load()
    _check(lib.pa_copy_blocks_fp8(
        _dev_ptr(k_cache, torch.uint8, "k_cache"), _dev_ptr(v_cache, torch.uint8, "v_cache"),
        _dev_ptr(pairs, torch.int32, "pairs"), pairs.shape[0], Hkv, D, BS, NB,
        _stream_handle(stream)), "pa_copy_blocks_fp8")


def _check_fp4_rows(k_rows, v_rows, k_cache, v_cache, slot_mapping, k_scale, v_scale, who: str):
    rows, cache = k_rows.shape, k_cache.shape
    T, Hkv, D = rows
    NB, Hkv2, BS, bytes_ = cache
    if D not in (64, 128) or bytes_ * 16 != D * 9 or Hkv2 != Hkv or v_rows.shape != rows \
            or v_cache.shape != cache or slot_mapping.shape != (T,) \
            or k_scale.numel() != Hkv or v_scale.numel() != Hkv:
        raise ValueError(f"shape mismatch in {who}")
    return T, Hkv, D, BS, NB


def pa_reshape_and_cache_fp4(k_new, v_new, k_cache, v_cache, slot_mapping, k_scale, v_scale,
                             stream=None) -> None:
    """KV write into the 4-bit cache (uint8, ``fp4_cache_shape``): E2M1 codes with
    an E4M3 scale per 16 elements and the float32 scale of each KV head."""
    import torch

    dims = _check_fp4_rows(k_new, v_new, k_cache, v_cache, slot_mapping, k_scale, v_scale,
                           "pa_reshape_and_cache_fp4")
    lib = load()
    _check(lib.pa_reshape_and_cache_fp4(
        _dev_ptr(k_new, torch.bfloat16, "k_new"), _dev_ptr(v_new, torch.bfloat16, "v_new"),
        _dev_ptr(k_cache, torch.uint8, "k_cache"), _dev_ptr(v_cache, torch.uint8, "v_cache"),
        _dev_ptr(slot_mapping, torch.int64, "slot_mapping"),
        _dev_ptr(k_scale, torch.float32, "k_scale"), _dev_ptr(v_scale, torch.float32, "v_scale"),
        *dims, _stream_handle(stream)), "pa_reshape_and_cache_fp4")


def pa_gather_fp4(k_cache, v_cache, slot_mapping, k_scale, v_scale, k_out=None, v_out=None,
                  stream=None):
    """Rows of the 4-bit cache read back as bf16 [num_tokens][Hkv][D]; returns
    (k_out, v_out). A negative slot gives a row of zeros."""
    import torch

    fmt, D = kv_cache_format(k_cache)
    if fmt != KV_FP4_E2M1:
        raise ValueError("pa_gather_fp4 reads a 4-bit cache")
    shape = (slot_mapping.shape[0], k_cache.shape[1], D)
    if k_out is None:
        k_out = _empty(stream, k_cache, shape, torch.bfloat16)
    if v_out is None:
        v_out = _empty(stream, k_cache, shape, torch.bfloat16)
    dims = _check_fp4_rows(k_out, v_out, k_cache, v_cache, slot_mapping, k_scale, v_scale,
                           "pa_gather_fp4")
    lib = load()
    _check(lib.pa_gather_fp4(
        _dev_ptr(k_cache, torch.uint8, "k_cache"), _dev_ptr(v_cache, torch.uint8, "v_cache"),
        _dev_ptr(k_out, torch.bfloat16, "k_out"), _dev_ptr(v_out, torch.bfloat16, "v_out"),
        _dev_ptr(slot_mapping, torch.int64, "slot_mapping"),
        _dev_ptr(k_scale, torch.float32, "k_scale"), _dev_ptr(v_scale, torch.float32, "v_scale"),
        *dims, _stream_handle(stream)), "pa_gather_fp4")
    return k_out, v_out


def pa_copy_blocks_fp4(k_cache, v_cache, pairs, stream=None) -> None:
    import torch

    fmt, D = kv_cache_format(k_cache)
    if fmt != KV_FP4_E2M1 or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("pa_copy_blocks_fp4 copies blocks of a 4-bit cache")
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be int32 [n][2]")
    NB, Hkv, BS, _ = k_cache.shape
    lib = load()
    _check(lib.pa_copy_blocks_fp4(
        _dev_ptr(k_cache, torch.uint8, "k_cache"), _dev_ptr(v_cache, torch.uint8, "v_cache"),
        _dev_ptr(pairs, torch.int32, "pairs"), pairs.shape[0], Hkv, D, BS, NB,
        _stream_handle(stream)), "pa_copy_blocks_fp4")


def make_token_weights_params(q, k_cache, block_tables, context_lens, max_context_len: int,
                              token_weights, accumulate: bool = True,
                              scale: Optional[float] = None, k_scale=None) -> TokenWeightsParams:
    """Marshal a pa_token_weights call: q bf16 [B][Hq][D] or [B][Q][Hq][D], a K
    cache of any type (``kv_cache_format``; uint8 ones need k_scale), token_weights
    float32 [B][stride]."""
    import torch

    if q.dim() == 4:
        B, QL, Hq, D = q.shape
    else:
        (B, Hq, D), QL = q.shape, 0
    fmt, D2 = kv_cache_format(k_cache)
    NB, Hkv, BS, _ = k_cache.shape
    if D2 != D:
        raise ValueError("q and k_cache differ in head_dim")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or context_lens.shape != (B,):
        raise ValueError("block_tables must be [num_seqs][max_blocks], context_lens [num_seqs]")
    if token_weights.dim() != 2 or token_weights.shape[0] != B:
        raise ValueError("token_weights must be [num_seqs][stride]")
    ks = None
    if fmt != KV_BF16:
        if k_scale is None or k_scale.numel() != Hkv:
            raise ValueError("the 8-bit and 4-bit caches need k_scale [num_kv_heads]")
        ks = _dev_ptr(k_scale, torch.float32, "k_scale")
    return TokenWeightsParams(
        _dev_ptr(q, torch.bfloat16, "q"),
        _dev_ptr(k_cache, torch.bfloat16 if fmt == KV_BF16 else torch.uint8, "k_cache"),
        _dev_ptr(block_tables, torch.int32, "block_tables"),
        _dev_ptr(context_lens, torch.int32, "context_lens"),
        _dev_ptr(token_weights, torch.float32, "token_weights"), token_weights.shape[1],
        block_tables.shape[1], B, Hq, Hkv, D, BS, NB, int(max_context_len),
        float(1.0 / math.sqrt(D) if scale is None else scale), fmt, ks, int(QL),
        int(bool(accumulate)))


def pa_token_weights_workspace_size(q, k_cache, block_tables, context_lens, max_context_len: int,
                                    token_weights, k_scale=None) -> int:
    """Workspace bytes of ``pa_token_weights`` for these arguments."""
    p = make_token_weights_params(q, k_cache, block_tables, context_lens, max_context_len,
                                  token_weights, k_scale=k_scale)
    return int(load().pa_token_weights_workspace_size(ctypes.byref(p)))


def pa_token_weights(q, k_cache, block_tables, context_lens, max_context_len: int, token_weights,
                     accumulate: bool = True, scale: Optional[float] = None, workspace=None,
                     stream=None, k_scale=None):
    """The attention weight that the new tokens give to every cached token, summed
    over query heads and new tokens, added to (or, without ``accumulate``,
    written over) ``token_weights`` [B][stride] for t < context_lens[b]; returns
    it. Reads K only."""
    import torch

    lib = load()
    p = make_token_weights_params(q, k_cache, block_tables, context_lens, max_context_len,
                                  token_weights, accumulate, scale, k_scale)
    if workspace is None:
        need = int(lib.pa_token_weights_workspace_size(ctypes.byref(p)))
        workspace = _empty(stream, q, max(need, 256), torch.uint8)
    _check(lib.pa_token_weights(ctypes.byref(p), _dev_ptr(workspace, torch.uint8, "workspace"),
                                workspace.numel(), _stream_handle(stream)), "pa_token_weights")
    return token_weights


def pa_evict_select(token_weights, context_lens, budget: int, recent: int = 0, keep=None,
                    new_lens=None, stream=None):
    """The tokens every sequence keeps under ``budget``: the last ``recent`` ones
    and those with the largest weights. Returns (keep int32 [B][budget], ascending,
    -1 behind; new_lens int32 [B])."""
    import torch

    if token_weights.dim() != 2 or context_lens.shape != (token_weights.shape[0],):
        raise ValueError("token_weights must be [num_seqs][stride], context_lens [num_seqs]")
    B = token_weights.shape[0]
    if keep is None:
        keep = _empty(stream, token_weights, (B, max(int(budget), 0)), torch.int32)
    if new_lens is None:
        new_lens = _empty(stream, token_weights, B, torch.int32)
    if keep.shape != (B, budget) or new_lens.shape != (B,):
        raise ValueError("keep must be [num_seqs][budget], new_lens [num_seqs]")
    _check(load().pa_evict_select(
        _dev_ptr(token_weights, torch.float32, "token_weights"),
        _dev_ptr(context_lens, torch.int32, "context_lens"), _dev_ptr(keep, torch.int32, "keep"),
        _dev_ptr(new_lens, torch.int32, "new_lens"), B, token_weights.shape[1], int(budget),
        int(recent), _stream_handle(stream)), "pa_evict_select")
    return keep, new_lens


def pa_evict_compact(k_cache, v_cache, block_tables, dst_tables, keep, new_lens,
                     token_weights=None, stream=None) -> None:
    """Move the kept tokens' rows: token keep[b][j] of ``block_tables`` becomes
    token j of ``dst_tables`` (which may be ``block_tables``), for j <
    new_lens[b]. ``token_weights`` is compacted along, zeroed behind."""
    import torch

    fmt, D = kv_cache_format(k_cache)
    NB, Hkv, BS, _ = k_cache.shape
    B = new_lens.shape[0]
    if not _v_cache_ok(fmt, k_cache, v_cache):
        raise ValueError("shape mismatch between k_cache and v_cache")
    if block_tables.dim() != 2 or dst_tables.dim() != 2 or keep.dim() != 2 \
            or block_tables.shape[0] != B or dst_tables.shape[0] != B or keep.shape[0] != B \
            or (token_weights is not None
                and (token_weights.dim() != 2 or token_weights.shape[0] != B)):
        raise ValueError("block_tables, dst_tables, keep and token_weights must be [num_seqs][...]")
    cache_dtype = torch.bfloat16 if fmt == KV_BF16 else torch.uint8
    p = EvictCompactParams(
        _dev_ptr(k_cache, cache_dtype, "k_cache"), _dev_ptr(v_cache, cache_dtype, "v_cache"),
        _dev_ptr(block_tables, torch.int32, "block_tables"),
        _dev_ptr(dst_tables, torch.int32, "dst_tables"), _dev_ptr(keep, torch.int32, "keep"),
        _dev_ptr(new_lens, torch.int32, "new_lens"),
        None if token_weights is None else _dev_ptr(token_weights, torch.float32, "token_weights"),
        0 if token_weights is None else token_weights.shape[1], block_tables.shape[1],
        dst_tables.shape[1], keep.shape[1], B, Hkv, D, BS, NB, fmt)
    _check(load().pa_evict_compact(ctypes.byref(p), _stream_handle(stream)), "pa_evict_compact")


def make_free_ring(blocks, num_blocks: int, device="cuda"):
    """A ring for ``pa_update_tables`` that holds the given free block ids (handed out in
    this order) and has room for every block of a cache of ``num_blocks``. Returns
    (free_ring int32 [num_blocks], ring_state int32 [4])."""
    import torch

    ids = np.asarray(list(blocks), dtype=np.int64)
    if num_blocks < 1 or ids.ndim != 1 or len(set(ids.tolist())) != len(ids) \
            or (len(ids) and (ids.min() < 0 or ids.max() >= num_blocks)):
        raise ValueError("blocks must be distinct ids in [0, num_blocks)")
    ring = np.full(num_blocks, -1, dtype=np.int32)
    ring[:len(ids)] = ids
    state = np.array([0, len(ids), 0, 0], dtype=np.int32)
    return torch.from_numpy(ring).to(device), torch.from_numpy(state).to(device)


_NO_ROWS = 256  # stands for the address of an array of no bytes


def pa_update_tables(block_tables, old_lens, new_lens, free_ring, ring_state, new_ring_state,
                     num_blocks: int, block_size: int, slot_mapping=None, positions=None,
                     token_starts=None, stream=None) -> None:
    """Tables on the device: row b of ``block_tables`` (int32 [B][max_blocks]), which
    holds blocks for ``old_lens[b]`` tokens, gets them for ``new_lens[b]`` from the ring
    of free blocks (``make_free_ring``), or gives the blocks behind back to it.
    ``slot_mapping`` (int64 [T]), ``positions`` (int32 [T]) and ``token_starts`` (int32
    [B + 1]) get the new tokens, packed, -1 behind; ``new_ring_state`` (int32 [4]) the
    ring's state: head, count, and 0 where the step was done (see the C header)."""
    dev = _current()
    tables, lens, ring = block_tables.shape, old_lens.shape, free_ring.shape
    if len(tables) != 2 or lens != tables[:1] or new_lens.shape != lens:
        raise ValueError("block_tables must be [num_seqs][max_blocks], the lengths [num_seqs]")
    if len(ring) != 1 or ring_state.shape != (4,) or new_ring_state.shape != (4,):
        raise ValueError("free_ring must be [ring_size], the states [4]")
    B = lens[0]
    slots = pos = starts = None
    T = 0
    # (torch has no address for a tensor without rows, and NULL would say that it is not wanted)
    if slot_mapping is not None:
        slots, rows = _ptr(slot_mapping, _i64, "slot_mapping", dev) or _NO_ROWS, slot_mapping.shape
        T = rows[0] if len(rows) == 1 else -1
    if positions is not None:
        pos, rows = _ptr(positions, _i32, "positions", dev) or _NO_ROWS, positions.shape
        T = rows[0] if len(rows) == 1 and (slots is None or rows[0] == T) else -1
    if token_starts is not None:
        starts = _ptr(token_starts, _i32, "token_starts", dev)
        T = T if token_starts.shape == (B + 1,) else -1
    if T < 0:
        raise ValueError("slot_mapping and positions must be [max_new_tokens], token_starts "
                         "[num_seqs + 1]")
    p = UpdateTablesParams(
        _ptr(block_tables, _i32, "block_tables", dev), _ptr(old_lens, _i32, "old_lens", dev),
        _ptr(new_lens, _i32, "new_lens", dev), _ptr(free_ring, _i32, "free_ring", dev),
        _ptr(ring_state, _i32, "ring_state", dev), _ptr(new_ring_state, _i32, "new_ring_state", dev),
        slots, pos, starts, tables[1], B, int(block_size), int(num_blocks), ring[0], T)
    _check(load().pa_update_tables(ctypes.byref(p), _stream_handle(stream)), "pa_update_tables")


def block_bounds_shape(num_blocks: int, num_kv_heads: int, head_dim: int):
    """Shape of the bounds of a cache's blocks (bf16): least and largest keys."""
    return (num_blocks, num_kv_heads, 2, head_dim)


def pa_block_bounds(k_cache, bounds, block_tables, context_lens, max_new_tokens: int,
                    old_lens=None, stream=None):
    """The least and the largest key, element by element, of every (block, KV head) that
    holds a token from ``old_lens[b]`` on (None: from the first), written into ``bounds``
    (bf16, ``block_bounds_shape``); returns it. K caches of every type; the head's scale
    is left out. ``max_new_tokens`` is an upper bound of ``context_lens - old_lens``."""
    dev = _current()
    fmt, D = kv_cache_format(k_cache)
    NB, Hkv, BS, _ = k_cache.shape
    tables = block_tables.shape
    if tuple(bounds.shape) != (NB, Hkv, 2, D):
        raise ValueError("bounds must be [num_blocks][num_kv_heads][2][head_dim]")
    if len(tables) != 2 or context_lens.shape != tables[:1] \
            or (old_lens is not None and old_lens.shape != tables[:1]):
        raise ValueError("block_tables must be [num_seqs][max_blocks], the lengths [num_seqs]")
    p = BlockBoundsParams(
        _ptr(k_cache, _bf16 if fmt == KV_BF16 else _u8, "k_cache", dev),
        _ptr(bounds, _bf16, "bounds", dev),
        _ptr(block_tables, _i32, "block_tables", dev),
        _ptr(context_lens, _i32, "context_lens", dev),
        None if old_lens is None else _ptr(old_lens, _i32, "old_lens", dev),
        tables[1], tables[0], Hkv, D, BS, NB, int(max_new_tokens), fmt)
    _check(load().pa_block_bounds(ctypes.byref(p), _stream_handle(stream)), "pa_block_bounds")
    return bounds


def pa_block_scores(q, bounds, block_tables, context_lens, max_context_len: int, block_size: int,
                    scores=None, scale: Optional[float] = None, k_scale=None, stream=None):
    """An upper bound (up to fp32 rounding) of the score that any key of a block reaches with
    any new token and query head of a KV head: float32 [B][Hkv][stride], of which the blocks of each
    sequence are written; returns it. q bf16 [B][Hq][D] or [B][Q][Hq][D]; ``k_scale`` is
    the head scale of the 8-bit and 4-bit caches."""
    dev = _current()
    shape = q.shape
    if len(shape) == 4:
        B, QL, Hq, D = shape
    else:
        (B, Hq, D), QL = shape, 0
    NB, Hkv, two, D2 = bounds.shape
    tables = block_tables.shape
    if two != 2 or D2 != D:
        raise ValueError("bounds must be [num_blocks][num_kv_heads][2][head_dim], head_dim as in q")
    if len(tables) != 2 or tables[0] != B or context_lens.shape != (B,):
        raise ValueError("block_tables must be [num_seqs][max_blocks], context_lens [num_seqs]")
    if k_scale is not None and k_scale.numel() != Hkv:
        raise ValueError("k_scale must be [num_kv_heads]")
    if scores is None:
        scores = _empty(stream, q, (B, Hkv, tables[1]), _f32)
    if scores.dim() != 3 or scores.shape[:2] != (B, Hkv):
        raise ValueError("scores must be [num_seqs][num_kv_heads][stride]")
    p = BlockScoresParams(
        _ptr(q, _bf16, "q", dev), _ptr(bounds, _bf16, "bounds", dev),
        None if k_scale is None else _ptr(k_scale, _f32, "k_scale", dev),
        _ptr(block_tables, _i32, "block_tables", dev),
        _ptr(context_lens, _i32, "context_lens", dev),
        _ptr(scores, _f32, "scores", dev), scores.shape[2], tables[1], B, Hq, Hkv, D,
        int(block_size), NB, int(max_context_len),
        float(1.0 / math.sqrt(D) if scale is None else scale), int(QL))
    _check(load().pa_block_scores(ctypes.byref(p), _stream_handle(stream)), "pa_block_scores")
    return scores


def pa_block_select(scores, context_lens, block_size: int, budget: int, sink: int = 1,
                    recent: int = 1, selected=None, stream=None):
    """The blocks that every (sequence, KV head) reads under ``budget``: the first ``sink``,
    the last ``recent`` and those with the largest scores. Returns ``selected`` (int32
    [B][Hkv][budget], ascending, -1 behind)."""
    dev = _current()
    if scores.dim() != 3 or context_lens.shape != scores.shape[:1]:
        raise ValueError("scores must be [num_seqs][num_kv_heads][stride], context_lens [num_seqs]")
    B, Hkv, stride = scores.shape
    if selected is None:
        selected = _empty(stream, scores, (B, Hkv, max(int(budget), 0)), _i32)
    if selected.shape != (B, Hkv, budget):
        raise ValueError("selected must be [num_seqs][num_kv_heads][budget]")
    _check(load().pa_block_select(
        _ptr(scores, _f32, "scores", dev),
        _ptr(context_lens, _i32, "context_lens", dev),
        _ptr(selected, _i32, "selected", dev), B, Hkv, stride, int(block_size), int(budget),
        int(sink), int(recent), _stream_handle(stream)), "pa_block_select")
    return selected


def _selected_shape(q, k_cache, selected) -> int:
    shape = selected.shape
    if len(shape) != 3 or shape[0] != q.shape[0] or shape[1] != k_cache.shape[1]:
        raise ValueError("selected must be [num_seqs][num_kv_heads][num_selected]")
    return shape[2]


def pa_decode_selected_workspace_size(q, k_cache, v_cache, block_tables, context_lens,
                                      max_context_len: int, selected, k_scale=None,
                                      v_scale=None) -> int:
    """Workspace bytes of ``pa_decode_selected`` for these arguments."""
    p = make_decode_params(q, q, k_cache, v_cache, block_tables, context_lens, max_context_len,
                           k_scale=k_scale, v_scale=v_scale)
    return int(load().pa_decode_selected_workspace_size(
        ctypes.byref(p), _selected_shape(q, k_cache, selected)))


def pa_decode_selected(q, k_cache, v_cache, block_tables, context_lens, max_context_len: int,
                       selected, scale: Optional[float] = None, out=None, workspace=None,
                       stream=None, k_scale=None, v_scale=None):
    """Paged decode attention over the blocks listed in ``selected`` (int32
    [B][Hkv][num_selected], logical blocks of the sequence, negative ones skipped) alone;
    returns ``out`` (bf16, the shape of ``q``). Caches of every type, one or several new
    tokens, as in ``pa_decode``. No workspace is needed; one that is given is not used."""
    dev = _current()
    lib = load()
    n = _selected_shape(q, k_cache, selected)
    if out is None:
        out = _empty(stream, q, q.shape, q.dtype)
    p = make_decode_params(q, out, k_cache, v_cache, block_tables, context_lens, max_context_len,
                           scale, k_scale=k_scale, v_scale=v_scale)
    ws_ptr = _ptr(workspace, _u8, "workspace", dev) if workspace is not None else None
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check(lib.pa_decode_selected(ctypes.byref(p), _ptr(selected, _i32, "selected", dev), n,
                                  ws_ptr, ws_bytes, _stream_handle(stream)), "pa_decode_selected")
    return out


def pa_device_errors(stream=None) -> int:
    flags = ctypes.c_uint32(0)
    _check(load().pa_device_errors(_stream_handle(stream), ctypes.byref(flags)), "pa_device_errors")
    return int(flags.value)


# --------------------------------------------------------------------------
# host block pool
# --------------------------------------------------------------------------

class Pool:
    """Host block pool (``pa_pool_*`` / ``pa_seq_*``). Free list is a stack seeded
    from ``free_order`` (first element handed out first)."""

    def __init__(self, num_blocks: int, block_size: int = 16,
                 free_order: Optional[Sequence[int]] = None):
        self._lib = load()
        self._h = ctypes.c_void_p()
        order = None
        if free_order is not None:
            order = np.ascontiguousarray(np.asarray(free_order, dtype=np.int32))
        _check(self._lib.pa_pool_create(num_blocks, block_size,
                                        None if order is None else order.ctypes.data,
                                        ctypes.byref(self._h)), "pa_pool_create")
        self.num_blocks = num_blocks
        self.block_size = block_size

    def close(self) -> None:
        if self._h:
            self._lib.pa_pool_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def alloc(self) -> int:
        b = ctypes.c_int32()
        _check(self._lib.pa_pool_alloc(self._h, ctypes.byref(b)), "pa_pool_alloc")
        return b.value

    def incref(self, blk: int) -> None:
        _check(self._lib.pa_pool_incref(self._h, blk), "pa_pool_incref")

    def decref(self, blk: int) -> None:
        _check(self._lib.pa_pool_decref(self._h, blk), "pa_pool_decref")

    def refcount(self, blk: int) -> int:
        return int(self._lib.pa_pool_refcount(self._h, blk))

    def stats(self) -> dict:
        st = PoolStats()
        _check(self._lib.pa_pool_stats(self._h, ctypes.byref(st)), "pa_pool_stats")
        return {n: getattr(st, n) for n, _ in PoolStats._fields_}

    def seq_create(self) -> int:
        s = ctypes.c_int32()
        _check(self._lib.pa_seq_create(self._h, ctypes.byref(s)), "pa_seq_create")
        return s.value

    def seq_free(self, seq: int) -> None:
        _check(self._lib.pa_seq_free(self._h, seq), "pa_seq_free")

    def seq_fork(self, parent: int, num_tokens: int) -> int:
        c = ctypes.c_int32()
        _check(self._lib.pa_seq_fork(self._h, parent, num_tokens, ctypes.byref(c)), "pa_seq_fork")
        return c.value

    def append_slot(self, seq: int) -> Tuple[int, Optional[Tuple[int, int]]]:
        slot = ctypes.c_int64()
        pair = (ctypes.c_int32 * 2)()
        has = ctypes.c_int32()
        _check(self._lib.pa_seq_append_slot(self._h, seq, ctypes.byref(slot), pair,
                                            ctypes.byref(has)), "pa_seq_append_slot")
        return slot.value, ((pair[0], pair[1]) if has.value else None)

    def append_tokens(self, seq: int, n: int, want_slots: bool = True):
        slots = np.empty(max(n, 1), dtype=np.int64)
        pairs = np.empty((max(n, 1), 2), dtype=np.int32)
        ncow = ctypes.c_int32()
        _check(self._lib.pa_seq_append_tokens(
            self._h, seq, n, slots.ctypes.data if want_slots else None, pairs.ctypes.data,
            ctypes.byref(ncow)), "pa_seq_append_tokens")
        return (slots[:n].tolist() if want_slots else None,
                [tuple(int(x) for x in r) for r in pairs[:ncow.value]])

    def length(self, seq: int) -> int:
        n = ctypes.c_int32()
        _check(self._lib.pa_seq_length(self._h, seq, ctypes.byref(n)), "pa_seq_length")
        return n.value

    def table(self, seq: int) -> List[int]:
        n = ctypes.c_int32()
        _check(self._lib.pa_seq_table(self._h, seq, None, 0, ctypes.byref(n)), "pa_seq_table")
        buf = np.empty(max(n.value, 1), dtype=np.int32)
        _check(self._lib.pa_seq_table(self._h, seq, buf.ctypes.data, buf.shape[0],
                                      ctypes.byref(n)), "pa_seq_table")
        return buf[:n.value].tolist()

    def compact(self, seqs: Sequence[int], new_lens: Sequence[int]) -> None:
        """Shorten the sequences in blocks they may write (for ``pa_evict_compact``:
        export the tables before and after)."""
        s = np.ascontiguousarray(np.asarray(seqs, dtype=np.int32))
        n = np.ascontiguousarray(np.asarray(new_lens, dtype=np.int32))
        if s.shape != n.shape or s.ndim != 1:
            raise ValueError("seqs and new_lens must be lists of the same length")
        _check(self._lib.pa_pool_compact(self._h, s.ctypes.data, n.ctypes.data, len(s)),
               "pa_pool_compact")

    def export(self, seqs: Sequence[int], max_blocks: int):
        s = np.ascontiguousarray(np.asarray(seqs, dtype=np.int32))
        tables = np.empty((len(s), max_blocks), dtype=np.int32)
        lens = np.empty(len(s), dtype=np.int32)
        _check(self._lib.pa_pool_export(self._h, s.ctypes.data, len(s), max_blocks,
                                        tables.ctypes.data, lens.ctypes.data), "pa_pool_export")
        return tables, lens

    def create_prompt(self, tokens: Sequence[int]):
        """New sequence holding a prompt, its leading full blocks mapped from the
        prefix cache. Returns (seq, cached_tokens, slots)."""
        t = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
        seq, cached = ctypes.c_int32(), ctypes.c_int32()
        slots = np.empty(max(len(t), 1), dtype=np.int64)
        _check(self._lib.pa_seq_create_prompt(self._h, t.ctypes.data if len(t) else None, len(t),
                                              ctypes.byref(seq), ctypes.byref(cached),
                                              slots.ctypes.data), "pa_seq_create_prompt")
        return seq.value, cached.value, slots[:len(t)].tolist()

    def prefix_stats(self) -> dict:
        st = PrefixStats()
        _check(self._lib.pa_pool_prefix_stats(self._h, ctypes.byref(st)), "pa_pool_prefix_stats")
        return {"cached_blocks": st.cached_blocks, "evictable_blocks": st.evictable_blocks,
                "lookups": st.lookups, "hits": st.hits}
