"""Paged MLA decode for GB300 — thin Python binding over the libmla C ABI.

The binding only marshals arguments: it checks tensor dtypes/devices/shapes
(raising ValueError that names the argument, the MAX kernel-wrapper
convention), allocates outputs and scratch with torch when the caller does
not pass them, and calls the C entry points on the current CUDA stream.
Every step of decode runs in the library's CUDA kernels; there is no other
code path.  If ``libmla.so`` has not been built, every call raises.

    sched, num_splits = get_metadata(cache_seqlens, h_q=..., s_q=..., topk=..., is_fp8=...)
    out, lse = decode(q, kvcache, block_table, cache_seqlens, sm_scale,
                      sched, num_splits, is_causal=..., indices=...)
    out, lse = sparse_prefill(q, kv, indices, sm_scale)

    lens, row_offsets, slots, cursor = assign_pages(cache_lengths, new_tokens, free_pages, free_cursor,
                                                    block_table, num_tokens)
    cache_store(latent, rope, slots, kvcache)
    out, lse = window_decode(q, kvcache, block_table, lens, sm_scale, window=..., sinks=...)
    out, lse = shared_prefix_decode(q, kvcache, prefix_table, prefix_length, block_table, lens, sm_scale)
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import operator
import os
import threading
import warnings
from typing import Optional, Tuple

import torch

from . import builder as _build

D_QK = 576
D_V = 512
PAGE_SIZE = 64
FP8_ROW_BYTES = 656
MAX_PAGES = (2 ** 31 - 1) // PAGE_SIZE  # slots are int32

MLA_OK = 0
STATUS_NAMES = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_WORKSPACE",
                4: "MLA_ERR_CUDA", 5: "MLA_ERR_DEVICE_BOUNDS", 6: "MLA_ERR_DEVICE_TIMEOUT"}
DEVICE_BAD_PAGE = 0x1
DEVICE_TIMEOUT = 0x2
DEVICE_BAD_SCHEDULE = 0x4
DEVICE_NO_ROOM = 0x8

_lock = threading.Lock()
_lib = None
_native = None  # csrc/binding.cpp, loaded with the library (if it was built)


class MLAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class DecodeArgs(ctypes.Structure):
    """Mirror of ``mla_decode_args`` in include/mla.h."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("batch", ctypes.c_int), ("s_q", ctypes.c_int), ("h_q", ctypes.c_int),
        ("kvcache", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
        ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int),
        ("cache_seqlens", ctypes.c_void_p), ("sm_scale", ctypes.c_float), ("is_causal", ctypes.c_int),
        ("is_fp8", ctypes.c_int), ("indices", ctypes.c_void_p), ("topk", ctypes.c_int),
        ("sched", ctypes.c_void_p), ("num_splits", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("kv_scales", ctypes.c_void_p), ("topk_lengths", ctypes.c_void_p),
    ]


class SparsePrefillArgs(ctypes.Structure):
    """Mirror of ``mla_sparse_prefill_args`` in include/mla.h."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("s_q", ctypes.c_int), ("h_q", ctypes.c_int),
        ("kv", ctypes.c_void_p), ("s_kv", ctypes.c_int),
        ("indices", ctypes.c_void_p), ("topk", ctypes.c_int), ("sm_scale", ctypes.c_float),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
    ]


class IndexTopkArgs(ctypes.Structure):
    """Mirror of ``mla_index_topk_args`` in include/mla.h."""
    _fields_ = [
        ("q_codes", ctypes.c_void_p), ("q_scales", ctypes.c_void_p), ("weights", ctypes.c_void_p),
        ("num_tokens", ctypes.c_int), ("h_idx", ctypes.c_int), ("row_offsets", ctypes.c_void_p),
        ("batch", ctypes.c_int), ("max_new_tokens", ctypes.c_int), ("k_codes", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
        ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int),
        ("cache_seqlens", ctypes.c_void_p), ("relu", ctypes.c_int), ("topk", ctypes.c_int),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("indices", ctypes.c_void_p),
    ]


class AssignPagesArgs(ctypes.Structure):
    """Mirror of ``mla_assign_pages_args`` in include/mla.h."""
    _fields_ = [
        ("cache_lengths", ctypes.c_void_p), ("new_tokens", ctypes.c_void_p), ("batch", ctypes.c_int),
        ("free_pages", ctypes.c_void_p), ("num_free", ctypes.c_int), ("free_cursor", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int), ("num_pages", ctypes.c_int),
        ("num_tokens", ctypes.c_int), ("cache_seqlens", ctypes.c_void_p), ("row_offsets", ctypes.c_void_p),
        ("slot_map", ctypes.c_void_p), ("next_cursor", ctypes.c_void_p),
    ]


class CacheStoreArgs(ctypes.Structure):
    """Mirror of ``mla_cache_store_args`` in include/mla.h."""
    _fields_ = [
        ("latent", ctypes.c_void_p), ("latent_stride", ctypes.c_int64), ("rope", ctypes.c_void_p),
        ("rope_stride", ctypes.c_int64), ("slot_map", ctypes.c_void_p), ("num_tokens", ctypes.c_int),
        ("kvcache", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
        ("is_fp8", ctypes.c_int), ("kv_scales", ctypes.c_void_p),
    ]


class WindowDecodeArgs(ctypes.Structure):
    """Mirror of ``mla_window_decode_args`` in include/mla.h."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("batch", ctypes.c_int), ("s_q", ctypes.c_int), ("h_q", ctypes.c_int),
        ("kvcache", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
        ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int),
        ("cache_seqlens", ctypes.c_void_p), ("sm_scale", ctypes.c_float), ("window", ctypes.c_int),
        ("sinks", ctypes.c_int), ("is_fp8", ctypes.c_int), ("kv_scales", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p),
    ]


class SharedPrefixDecodeArgs(ctypes.Structure):
    """Mirror of ``mla_shared_prefix_decode_args`` in include/mla.h."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("batch", ctypes.c_int), ("s_q", ctypes.c_int), ("h_q", ctypes.c_int),
        ("kvcache", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
        ("prefix_table", ctypes.c_void_p), ("prefix_table_len", ctypes.c_int), ("prefix_length", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int),
        ("cache_seqlens", ctypes.c_void_p), ("sm_scale", ctypes.c_float), ("is_causal", ctypes.c_int),
        ("is_fp8", ctypes.c_int), ("kv_scales", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
    ]


def library_path() -> str:
    return _build.LIB


def _load_binding():
    """The native binding, or None: then every call goes through ctypes."""
    try:
        spec = importlib.util.spec_from_file_location("_mla_binding", _build.BINDING)
        native = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(native)
        return native
    except (ImportError, OSError) as e:
        warnings.warn(f"the native binding is not used, calls go through ctypes ({e}): run "
                      "paged_mla_decode_07_gb300.build()", RuntimeWarning, stacklevel=3)
        return None


def lib():
    """Load libmla.so (built in-tree by ``build()``); raise if it is missing."""
    global _lib, _native
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(f"libmla.so not found at {path}: run paged_mla_decode_07_gb300.build.build()")
            L = ctypes.CDLL(path)
            I, P, S = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
            L.mla_abi_version.restype = I
            L.mla_last_error.restype = ctypes.c_char_p
            L.mla_metadata_size.argtypes = [I, I, I, I, I, ctypes.POINTER(I), ctypes.POINTER(I)]
            L.mla_metadata_size.restype = I
            L.mla_workspace_size.argtypes = [I, I, I, I, I, ctypes.POINTER(S)]
            L.mla_workspace_size.restype = I
            L.mla_get_metadata.argtypes = [P, I, I, I, I, I, P, P, P]
            L.mla_get_metadata.restype = I
            L.mla_test_hooks.argtypes = [I, I]
            L.mla_test_hooks.restype = I
            L.mla_decode.argtypes = [ctypes.POINTER(DecodeArgs), P]
            L.mla_decode.restype = I
            L.mla_get_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
            L.mla_fp8_cache_store.argtypes = [P, I, P, P, I, P, I, P, I, I, P]
            L.mla_fp8_cache_store.restype = I
            L.mla_get_device_status.restype = I
            L.mla_sparse_prefill_workspace_size.argtypes = [I, I, I, ctypes.POINTER(S)]
            L.mla_sparse_prefill_workspace_size.restype = I
            L.mla_sparse_prefill.argtypes = [ctypes.POINTER(SparsePrefillArgs), P]
            L.mla_sparse_prefill.restype = I
            L.mla_index_topk_workspace_size.argtypes = [I, I, ctypes.POINTER(S)]
            L.mla_index_topk_workspace_size.restype = I
            L.mla_index_topk.argtypes = [ctypes.POINTER(IndexTopkArgs), P]
            L.mla_index_topk.restype = I
            L.mla_assign_pages.argtypes = [ctypes.POINTER(AssignPagesArgs), P]
            L.mla_assign_pages.restype = I
            L.mla_cache_store.argtypes = [ctypes.POINTER(CacheStoreArgs), P]
            L.mla_cache_store.restype = I
            L.mla_window_decode_workspace_size.argtypes = [I, I, I, I, ctypes.POINTER(S)]
            L.mla_window_decode_workspace_size.restype = I
            L.mla_window_decode.argtypes = [ctypes.POINTER(WindowDecodeArgs), P]
            L.mla_window_decode.restype = I
            L.mla_shared_prefix_decode_workspace_size.argtypes = [I, I, I, I, I, ctypes.POINTER(S)]
            L.mla_shared_prefix_decode_workspace_size.restype = I
            L.mla_shared_prefix_decode.argtypes = [ctypes.POINTER(SharedPrefixDecodeArgs), P]
            L.mla_shared_prefix_decode.restype = I
            _native, _lib = _load_binding(), L
    return _lib


def _plain(name: str, *args):
    """The native binding's result for a call in its plain form, or None (see csrc/binding.cpp)."""
    if _native is None:
        lib()
        if _native is None:
            return None
    r = getattr(_native, name)(*args)
    if type(r) is int:
        _check(r)
    return r


def _int32(value, name: str) -> int:
    value = operator.index(value)
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{name} = {value} does not fit 32 bits")
    return value


def last_error() -> str:
    return lib().mla_last_error().decode()


def _check(status: int):
    if status != MLA_OK:
        msg = last_error()
        if status in (1, 2, 3):
            raise ValueError(f"{STATUS_NAMES[status]}: {msg}")
        raise MLAError(status, msg)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t, name, dtype, device=None, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype} (got {t.dtype})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions (got {tuple(t.shape)})")
    if ndim is not None and max(t.shape, default=0) >= 2 ** 31:  # (ctypes would cut the size off)
        raise ValueError(f"a dimension of {name} does not fit 32 bits (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class _On:
    """The device of a call's tensors and the stream it runs on, current while the call allocates
    and launches: memory that the call allocates then belongs to that stream in torch's allocator,
    so it is not handed out again while the call's kernels still use it."""
    __slots__ = ("handle", "ctx")

    def __init__(self, dev, stream):
        self.ctx = []
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=dev)
            if stream.device != dev:
                raise ValueError(f"stream must belong to {dev} (got {stream.device})")
            self.ctx.append(torch.cuda.stream(stream))
            self.handle = stream.cuda_stream
        else:
            self.handle = torch.cuda.current_stream(dev).cuda_stream
            if dev.index != torch.cuda.current_device():
                self.ctx.append(torch.cuda.device(dev))

    def __enter__(self):
        for c in self.ctx:
            c.__enter__()
        return ctypes.c_void_p(self.handle)

    def __exit__(self, *exc):
        for c in reversed(self.ctx):
            c.__exit__(*exc)


# the current stream's handle without the Stream object around it (a third of the binding's time in short calls)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(dev, stream, call):
    """call(stream handle) with the device of the tensors current, on `stream` or its current stream."""
    if stream is None and dev.index == torch.cuda.current_device():
        return call(_raw_stream(dev.index))
    with _On(dev, stream) as handle:
        return call(handle)


def _cuda_tensor(t, name):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _cache_format(kvcache, kv_scales, dev):
    """(is_fp8) of a paged cache after checking its type, shape and scales."""
    if kvcache.dtype == torch.uint8:
        _need(kvcache, "kvcache", torch.uint8, dev, 4)
        row = 640 if kv_scales is not None else FP8_ROW_BYTES
        if kvcache.shape[-1] != row or kvcache.shape[2] != 1:
            raise ValueError(f"FP8 kvcache must be [pages, page_size, 1, {row}] (got {tuple(kvcache.shape)})")
        if kv_scales is not None:
            _need(kv_scales, "kv_scales", torch.float32, dev)
            if kv_scales.numel() != kvcache.shape[0] * kvcache.shape[1]:
                raise ValueError("kv_scales must hold one scale per cached token")
        return True
    _need(kvcache, "kvcache", torch.bfloat16, dev, 4)
    if kvcache.shape[-1] != D_QK or kvcache.shape[2] != 1:
        raise ValueError(f"bf16 kvcache must be [pages, page_size, 1, {D_QK}] (got {tuple(kvcache.shape)})")
    if kv_scales is not None:
        raise ValueError("kv_scales given with a bf16 kvcache")
    return False


def metadata_size(batch: int, *, h_q: int, s_q: int, topk: int, is_fp8: bool) -> Tuple[int, int]:
    """(sched int32 elements, num_splits int32 elements) for one decode configuration."""
    a, b = ctypes.c_int(), ctypes.c_int()
    _check(lib().mla_metadata_size(batch, h_q, s_q, topk, int(bool(is_fp8)), ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def workspace_size(batch: int, *, h_q: int, s_q: int, topk: int, is_fp8: bool) -> int:
    """Scratch bytes mla_decode needs for one decode configuration."""
    n = ctypes.c_size_t()
    _check(lib().mla_workspace_size(batch, h_q, s_q, topk, int(bool(is_fp8)), ctypes.byref(n)))
    return n.value


def get_metadata(cache_seqlens: torch.Tensor, *, h_q: int, s_q: int, topk: int, is_fp8: bool, stream=None,
                 sched: Optional[torch.Tensor] = None, num_splits: Optional[torch.Tensor] = None):
    """Tile schedule for one decode step; reuse it for every layer of the step.  The keywords name
    the decode configuration (topk = 0: dense; is_fp8: the cache format) that decode() will run."""
    _need(cache_seqlens, "cache_seqlens", torch.int32, ndim=1)
    if not cache_seqlens.is_cuda:
        raise ValueError("cache_seqlens must be a CUDA tensor")
    dev = cache_seqlens.device
    batch = cache_seqlens.shape[0]
    ns, nn = metadata_size(batch, h_q=h_q, s_q=s_q, topk=topk, is_fp8=is_fp8)
    if sched is None:
        sched = torch.empty(ns, dtype=torch.int32, device=dev)
    if num_splits is None:
        num_splits = torch.empty(nn, dtype=torch.int32, device=dev)
    if sched.numel() < ns or num_splits.numel() < nn:
        raise ValueError("sched / num_splits buffers are too small")
    _check(lib().mla_get_metadata(ctypes.c_void_p(cache_seqlens.data_ptr()), batch, h_q, s_q, topk,
                                  int(bool(is_fp8)), ctypes.c_void_p(sched.data_ptr()),
                                  ctypes.c_void_p(num_splits.data_ptr()), _stream(stream)))
    return sched, num_splits


def set_test_hooks(num_parts: int = 0, debug_stall: bool = False) -> None:
    """Library test hooks (mla_test_hooks): force the schedule's part count (0 = default) and make
    the decode kernel's softmax role stall so that its bounded wait runs out."""
    _check(lib().mla_test_hooks(int(num_parts), int(bool(debug_stall))))


def decode(q: torch.Tensor, kvcache: torch.Tensor, block_table: torch.Tensor, cache_seqlens: torch.Tensor,
           sm_scale: float, sched: torch.Tensor, num_splits: torch.Tensor, is_causal: bool = False,
           indices: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
           lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None,
           kv_scales: Optional[torch.Tensor] = None, topk_lengths: Optional[torch.Tensor] = None):
    """Paged MLA decode.  Returns (out bf16 [b, s_q, h_q, 512], lse fp32 [b, s_q, h_q], base 2).
    kv_scales (fp32 [num_pages, 64]) selects the FP8 cache with one scale per token (640-byte rows);
    topk_lengths (int32 [b, s_q]) limits each sparse row to its first index slots."""
    _need(q, "q", torch.bfloat16, ndim=4)
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    dev = q.device
    batch, s_q, h_q, d = q.shape
    if d != D_QK:
        raise ValueError(f"q must have last dimension {D_QK} (got {d})")
    is_fp8 = kvcache.dtype == torch.uint8
    if is_fp8:
        _need(kvcache, "kvcache", torch.uint8, dev, 4)
        row = 640 if kv_scales is not None else FP8_ROW_BYTES
        if kvcache.shape[-1] != row or kvcache.shape[2] != 1:
            raise ValueError(f"FP8 kvcache must be [pages, page_size, 1, {row}]")
        if kv_scales is not None:
            _need(kv_scales, "kv_scales", torch.float32, dev)
            if kv_scales.numel() != kvcache.shape[0] * kvcache.shape[1]:
                raise ValueError("kv_scales must hold one scale per cached token")
    else:
        _need(kvcache, "kvcache", torch.bfloat16, dev, 4)
        if kvcache.shape[-1] != D_QK or kvcache.shape[2] != 1:
            raise ValueError(f"bf16 kvcache must be [pages, page_size, 1, {D_QK}]")
    _need(block_table, "block_table", torch.int32, dev, 2)
    _need(cache_seqlens, "cache_seqlens", torch.int32, dev, 1)
    if block_table.shape[0] != batch or cache_seqlens.shape[0] != batch:
        raise ValueError("block_table and cache_seqlens must have batch rows")
    topk = 0
    if indices is not None:
        _need(indices, "indices", torch.int32, dev, 3)
        if tuple(indices.shape[:2]) != (batch, s_q):
            raise ValueError(f"indices must be [batch, s_q, topk] (got {tuple(indices.shape)})")
        topk = indices.shape[2]
    if topk_lengths is not None:
        _need(topk_lengths, "topk_lengths", torch.int32, dev)
        if topk_lengths.numel() != batch * s_q:
            raise ValueError("topk_lengths must be [batch, s_q]")
    _need(sched, "sched", torch.int32, dev)
    _need(num_splits, "num_splits", torch.int32, dev)
    if out is None:
        out = torch.empty((batch, s_q, h_q, D_V), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((batch, s_q, h_q), dtype=torch.float32, device=dev)
    _need(out, "out", torch.bfloat16, dev)
    _need(lse, "lse", torch.float32, dev)
    if out.numel() != batch * s_q * h_q * D_V or lse.numel() != batch * s_q * h_q:
        raise ValueError("out / lse have the wrong size")
    if workspace is None:
        workspace = torch.empty(max(workspace_size(batch, h_q=h_q, s_q=s_q, topk=topk, is_fp8=is_fp8), 256),
                                dtype=torch.uint8, device=dev)
    a = DecodeArgs()
    a.q = q.data_ptr()
    a.batch, a.s_q, a.h_q = batch, s_q, h_q
    a.kvcache = kvcache.data_ptr()
    a.num_pages, a.page_size = kvcache.shape[0], kvcache.shape[1]
    a.block_table = block_table.data_ptr()
    a.block_table_stride = block_table.shape[1]
    a.cache_seqlens = cache_seqlens.data_ptr()
    a.sm_scale = float(sm_scale)
    a.is_causal = int(bool(is_causal))
    a.is_fp8 = int(is_fp8)
    a.indices = indices.data_ptr() if indices is not None else None
    a.topk = topk
    a.sched = sched.data_ptr()
    a.num_splits = num_splits.data_ptr()
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    a.out = out.data_ptr()
    a.lse = lse.data_ptr()
    a.kv_scales = kv_scales.data_ptr() if kv_scales is not None else None
    a.topk_lengths = topk_lengths.data_ptr() if topk_lengths is not None else None
    _check(lib().mla_decode(ctypes.byref(a), _stream(stream)))
    return out.view(batch, s_q, h_q, D_V), lse.view(batch, s_q, h_q)


def fp8_cache_store(x: torch.Tensor, input_row_offsets: torch.Tensor, cache_lengths: torch.Tensor,
                    block_table: torch.Tensor, kvcache: torch.Tensor, stream=None) -> None:
    """Quantise new tokens into the FP8 cache rows (mla_fp8_cache_store).

    x bf16 [num_tokens, 576]; input_row_offsets int32 [batch + 1]; cache_lengths int32 [batch];
    block_table int32 [batch, stride]; kvcache uint8 [num_pages, 64, 1, 656] (written in place).
    """
    if not torch.is_tensor(x) or x.device.type != "cuda":
        raise ValueError("x must be a CUDA tensor")
    dev = x.device
    _need(x, "x", torch.bfloat16, dev, 2)
    if x.shape[1] != 576:
        raise ValueError(f"x must be [num_tokens, 576] (got {tuple(x.shape)})")
    _need(input_row_offsets, "input_row_offsets", torch.int32, dev, 1)
    _need(cache_lengths, "cache_lengths", torch.int32, dev, 1)
    _need(block_table, "block_table", torch.int32, dev, 2)
    _need(kvcache, "kvcache", torch.uint8, dev, 4)
    batch = cache_lengths.shape[0]
    if input_row_offsets.shape[0] != batch + 1 or block_table.shape[0] != batch:
        raise ValueError("input_row_offsets must have batch + 1 entries and block_table batch rows")
    if kvcache.shape[2] != 1 or kvcache.shape[3] != 656:
        raise ValueError(f"kvcache must be [num_pages, page_size, 1, 656] (got {tuple(kvcache.shape)})")
    _check(lib().mla_fp8_cache_store(x.data_ptr(), x.shape[0], input_row_offsets.data_ptr(),
                                     cache_lengths.data_ptr(), batch, block_table.data_ptr(),
                                     block_table.shape[1], kvcache.data_ptr(), kvcache.shape[0], kvcache.shape[1],
                                     _stream(stream)))


def assign_pages(cache_lengths: torch.Tensor, new_tokens: torch.Tensor, free_pages: torch.Tensor,
                 free_cursor: torch.Tensor, block_table: torch.Tensor, num_tokens: int,
                 num_pages: Optional[int] = None, cache_seqlens: Optional[torch.Tensor] = None,
                 row_offsets: Optional[torch.Tensor] = None, slot_map: Optional[torch.Tensor] = None,
                 next_cursor: Optional[torch.Tensor] = None, stream=None):
    """Pages and slots of one step's new tokens (mla_assign_pages).

    cache_lengths, new_tokens int32 [batch]; free_pages int32 [num_free], used from entry free_cursor
    (int32 [1]) on; block_table int32 [batch, stride], its new entries written in place; num_tokens:
    the entries of the slot map, the new tokens of all requests or more (a padded step); num_pages:
    the cache's pages, to check page ids against.  Returns (cache_seqlens int32 [batch], row_offsets
    int32 [batch + 1], slot_map int32 [num_tokens], next_cursor int32 [1]); cache_seqlens may be
    given as cache_lengths and next_cursor as free_cursor, to advance them in place.
    """
    if stream is None:
        r = _plain("assign_pages", cache_lengths, new_tokens, free_pages, free_cursor, block_table, num_tokens, num_pages,
                   cache_seqlens, row_offsets, slot_map, next_cursor)
        if r is not None:
            return r
    dev = _cuda_tensor(cache_lengths, "cache_lengths")
    _need(cache_lengths, "cache_lengths", torch.int32, dev, 1)
    _need(new_tokens, "new_tokens", torch.int32, dev, 1)
    _need(free_pages, "free_pages", torch.int32, dev, 1)
    _need(free_cursor, "free_cursor", torch.int32, dev, 1)
    _need(block_table, "block_table", torch.int32, dev, 2)
    batch, num_tokens = cache_lengths.shape[0], _int32(num_tokens, "num_tokens")
    if new_tokens.shape[0] != batch or block_table.shape[0] != batch or free_cursor.shape[0] != 1:
        raise ValueError("new_tokens and block_table must have batch rows and free_cursor one entry")
    if num_tokens < 0:
        raise ValueError(f"num_tokens must be >= 0 (got {num_tokens})")
    sizes = (num_tokens, batch, batch + 1, 1)
    given = (slot_map, cache_seqlens, row_offsets, next_cursor)
    for t, name, n in zip(given, ("slot_map", "cache_seqlens", "row_offsets", "next_cursor"), sizes):
        if t is not None:
            _need(t, name, torch.int32, dev, 1)
            if t.shape[0] != n:
                raise ValueError(f"{name} must have {n} entries (got {t.shape[0]})")

    def call(handle):
        slots, lens, offsets, cursor = [torch.empty(n, dtype=torch.int32, device=dev) if t is None else t
                                        for t, n in zip(given, sizes)]
        a = AssignPagesArgs(cache_lengths.data_ptr(), new_tokens.data_ptr(), batch, free_pages.data_ptr(),
                            free_pages.shape[0], free_cursor.data_ptr(), block_table.data_ptr(),
                            block_table.shape[1], MAX_PAGES if num_pages is None else _int32(num_pages, "num_pages"), num_tokens,
                            lens.data_ptr(), offsets.data_ptr(), slots.data_ptr(), cursor.data_ptr())
        _check(lib().mla_assign_pages(ctypes.byref(a), handle))
        return lens, offsets, slots, cursor

    return _launch(dev, stream, call)


def cache_store(latent: torch.Tensor, rope: torch.Tensor, slot_map: torch.Tensor, kvcache: torch.Tensor,
                kv_scales: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write new tokens into the cache rows that slot_map names (mla_cache_store).

    latent bf16 [num_tokens, 512] and rope bf16 [num_tokens, 64], each with any row stride that is a
    multiple of 8 values (so both may be slices of one projection); slot_map int32 [num_tokens]
    (page * 64 + slot, negative: skipped), the slots distinct; kvcache bf16 [num_pages, 64, 1, 576],
    uint8 [.., 656] or, with kv_scales fp32 [num_pages, 64], uint8 [.., 640]; written in place.
    """
    if stream is None and _plain("cache_store", latent, rope, slot_map, kvcache, kv_scales):
        return
    dev = _cuda_tensor(latent, "latent")
    n = latent.shape[0] if latent.dim() == 2 else -1
    for t, name, width in ((latent, "latent", D_V), (rope, "rope", D_QK - D_V)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.device != dev:
            raise ValueError(f"{name} must be a bfloat16 tensor on {dev}")
        if t.dim() != 2 or t.shape[0] != n or t.shape[1] != width:
            raise ValueError(f"{name} must be [num_tokens, {width}] (got {tuple(t.shape)})")
        if t.stride(1) != 1:
            raise ValueError(f"the values of a row of {name} must be contiguous")
    _need(slot_map, "slot_map", torch.int32, dev, 1)
    if slot_map.shape[0] != n:
        raise ValueError(f"slot_map must have {n} entries (got {slot_map.shape[0]})")
    if not isinstance(kvcache, torch.Tensor):
        raise ValueError("kvcache must be a torch.Tensor")
    is_fp8 = _cache_format(kvcache, kv_scales, dev)
    a = CacheStoreArgs(latent.data_ptr(), latent.stride(0) if n > 1 else D_V, rope.data_ptr(),
                       rope.stride(0) if n > 1 else D_V, slot_map.data_ptr(), n, kvcache.data_ptr(),
                       kvcache.shape[0], kvcache.shape[1], int(is_fp8),
                       kv_scales.data_ptr() if kv_scales is not None else None)
    _launch(dev, stream, lambda handle: _check(lib().mla_cache_store(ctypes.byref(a), handle)))


def sparse_prefill_workspace_size(s_q: int, h_q: int, topk: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().mla_sparse_prefill_workspace_size(s_q, h_q, topk, ctypes.byref(n)))
    return n.value


def sparse_prefill(q: torch.Tensor, kv: torch.Tensor, indices: torch.Tensor, sm_scale: float,
                   out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """Sparse prefill (mla_sparse_prefill).  q bf16 [s_q, h_q, 576]; kv bf16 [s_kv, 576] or
    [s_kv, 1, 576]; indices int32 [s_q, topk] or [s_q, 1, topk].  Returns (out bf16
    [s_q, h_q, 512], lse fp32 [s_q, h_q], base 2)."""
    if not torch.is_tensor(q) or q.device.type != "cuda":
        raise ValueError("q must be a CUDA tensor")
    dev = q.device
    _need(q, "q", torch.bfloat16, dev, 3)
    s_q, h_q, d = q.shape
    if d != D_QK:
        raise ValueError(f"q must have last dimension {D_QK} (got {d})")
    _need(kv, "kv", torch.bfloat16, dev)
    if kv.dim() == 3:
        if kv.shape[1] != 1:
            raise ValueError(f"kv must have one KV head (got {tuple(kv.shape)})")
        kv = kv.view(kv.shape[0], kv.shape[2])
    if kv.dim() != 2 or kv.shape[1] != D_QK:
        raise ValueError(f"kv must be [s_kv, {D_QK}] (got {tuple(kv.shape)})")
    _need(indices, "indices", torch.int32, dev)
    if indices.dim() == 3:
        if indices.shape[1] != 1:
            raise ValueError(f"indices must have one KV head (got {tuple(indices.shape)})")
        indices = indices.view(indices.shape[0], indices.shape[2])
    if indices.dim() != 2 or indices.shape[0] != s_q:
        raise ValueError(f"indices must be [s_q, topk] (got {tuple(indices.shape)})")
    topk = indices.shape[1]
    if out is None:
        out = torch.empty((s_q, h_q, D_V), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((s_q, h_q), dtype=torch.float32, device=dev)
    _need(out, "out", torch.bfloat16, dev)
    _need(lse, "lse", torch.float32, dev)
    if out.numel() != s_q * h_q * D_V or lse.numel() != s_q * h_q:
        raise ValueError("out / lse have the wrong size")
    if workspace is None:
        workspace = torch.empty(sparse_prefill_workspace_size(s_q, h_q, topk), dtype=torch.uint8, device=dev)
    a = SparsePrefillArgs()
    a.q = q.data_ptr()
    a.s_q, a.h_q = s_q, h_q
    a.kv = kv.data_ptr()
    a.s_kv = kv.shape[0]
    a.indices = indices.data_ptr()
    a.topk = topk
    a.sm_scale = float(sm_scale)
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    a.out = out.data_ptr()
    a.lse = lse.data_ptr()
    _check(lib().mla_sparse_prefill(ctypes.byref(a), _stream(stream)))
    return out.view(s_q, h_q, D_V), lse.view(s_q, h_q)


def _decode_io(q, kvcache, block_table, cache_seqlens, kv_scales):
    """Checks what the decode calls over a paged cache share; returns (device, is_fp8)."""
    dev = _cuda_tensor(q, "q")
    _need(q, "q", torch.bfloat16, dev, 4)
    if q.shape[3] != D_QK:
        raise ValueError(f"q must have last dimension {D_QK} (got {q.shape[3]})")
    if not isinstance(kvcache, torch.Tensor):
        raise ValueError("kvcache must be a torch.Tensor")
    is_fp8 = _cache_format(kvcache, kv_scales, dev)
    _need(block_table, "block_table", torch.int32, dev, 2)
    _need(cache_seqlens, "cache_seqlens", torch.int32, dev, 1)
    if block_table.shape[0] != q.shape[0] or cache_seqlens.shape[0] != q.shape[0]:
        raise ValueError("block_table and cache_seqlens must have batch rows")
    return dev, is_fp8


def _outputs(q, out, lse):
    batch, s_q, h_q, _ = q.shape
    for t, name, dtype, shape in ((out, "out", torch.bfloat16, (batch, s_q, h_q, D_V)),
                                  (lse, "lse", torch.float32, (batch, s_q, h_q))):
        if t is not None:
            _need(t, name, dtype, q.device)
            if t.numel() != math.prod(shape):
                raise ValueError(f"{name} has the wrong size")
    out = torch.empty((batch, s_q, h_q, D_V), dtype=torch.bfloat16, device=q.device) if out is None else \
        out.view(batch, s_q, h_q, D_V)
    lse = torch.empty((batch, s_q, h_q), dtype=torch.float32, device=q.device) if lse is None else \
        lse.view(batch, s_q, h_q)
    return out, lse


def _scratch(workspace, nbytes, dev):
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if not isinstance(workspace, torch.Tensor) or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace


def window_decode_workspace_size(batch: int, *, h_q: int, s_q: int, is_fp8: bool) -> int:
    """Scratch bytes of window_decode."""
    n = ctypes.c_size_t()
    _check(lib().mla_window_decode_workspace_size(batch, h_q, s_q, int(bool(is_fp8)), ctypes.byref(n)))
    return n.value


def window_decode(q: torch.Tensor, kvcache: torch.Tensor, block_table: torch.Tensor, cache_seqlens: torch.Tensor,
                  sm_scale: float, window: int, sinks: int = 0, kv_scales: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """Decode attention over the first ``sinks`` and the last ``window`` keys (mla_window_decode).

    Arguments as decode()'s; query token i of an element of length L sits at position L - s_q + i and
    sees key t <= that position if t < sinks or t > position - window.  Returns (out bf16
    [b, s_q, h_q, 512], lse fp32 [b, s_q, h_q], base 2)."""
    if stream is None:
        r = _plain("window_decode", q, kvcache, block_table, cache_seqlens, sm_scale, window, sinks, kv_scales, out, lse,
                   workspace)
        if r is not None:
            return r
    dev, is_fp8 = _decode_io(q, kvcache, block_table, cache_seqlens, kv_scales)
    batch, s_q, h_q, _ = q.shape

    def call(handle):
        o, z = _outputs(q, out, lse)
        n = ctypes.c_size_t()
        if workspace is None:
            _check(lib().mla_window_decode_workspace_size(batch, h_q, s_q, int(is_fp8), ctypes.byref(n)))
        ws = _scratch(workspace, n.value, dev)
        a = WindowDecodeArgs(q.data_ptr(), batch, s_q, h_q, kvcache.data_ptr(), kvcache.shape[0], kvcache.shape[1],
                             block_table.data_ptr(), block_table.shape[1], cache_seqlens.data_ptr(), float(sm_scale),
                             _int32(window, "window"), _int32(sinks, "sinks"), int(is_fp8),
                             kv_scales.data_ptr() if kv_scales is not None else None, ws.data_ptr(), ws.nbytes,
                             o.data_ptr(), z.data_ptr())
        _check(lib().mla_window_decode(ctypes.byref(a), handle))
        return o, z

    return _launch(dev, stream, call)


def shared_prefix_decode_workspace_size(batch: int, *, h_q: int, s_q: int, prefix_table_len: int,
                                        is_fp8: bool) -> int:
    """Scratch bytes of shared_prefix_decode."""
    n = ctypes.c_size_t()
    _check(lib().mla_shared_prefix_decode_workspace_size(batch, h_q, s_q, prefix_table_len, int(bool(is_fp8)),
                                                         ctypes.byref(n)))
    return n.value


def shared_prefix_decode(q: torch.Tensor, kvcache: torch.Tensor, prefix_table: torch.Tensor,
                         prefix_length: torch.Tensor, block_table: torch.Tensor, cache_seqlens: torch.Tensor,
                         sm_scale: float, is_causal: bool = False, kv_scales: Optional[torch.Tensor] = None,
                         out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """Decode attention of a batch that shares a prefix, read once for the batch (mla_shared_prefix_decode).

    prefix_table int32 [pages] and prefix_length int32 [1] (on the device) name the shared tokens,
    block_table and cache_seqlens each element's own; every query row attends to both.  Tables as wide
    as their longest entry: small calls are slower with wide ones, and over an FP8 cache each column of
    prefix_table takes 73,728 bytes of workspace.  Returns (out bf16 [b, s_q, h_q, 512], lse fp32
    [b, s_q, h_q], base 2)."""
    if stream is None:
        r = _plain("shared_prefix_decode", q, kvcache, prefix_table, prefix_length, block_table, cache_seqlens, sm_scale,
                   is_causal, kv_scales, out, lse, workspace)
        if r is not None:
            return r
    dev, is_fp8 = _decode_io(q, kvcache, block_table, cache_seqlens, kv_scales)
    _need(prefix_table, "prefix_table", torch.int32, dev, 1)
    _need(prefix_length, "prefix_length", torch.int32, dev, 1)
    if prefix_length.shape[0] != 1:
        raise ValueError("prefix_length must have one entry")
    batch, s_q, h_q, _ = q.shape

    def call(handle):
        o, z = _outputs(q, out, lse)
        n = ctypes.c_size_t()
        if workspace is None:
            _check(lib().mla_shared_prefix_decode_workspace_size(batch, h_q, s_q, prefix_table.shape[0], int(is_fp8),
                                                                 ctypes.byref(n)))
        ws = _scratch(workspace, n.value, dev)
        a = SharedPrefixDecodeArgs(q.data_ptr(), batch, s_q, h_q, kvcache.data_ptr(), kvcache.shape[0],
                                   kvcache.shape[1], prefix_table.data_ptr(), prefix_table.shape[0],
                                   prefix_length.data_ptr(), block_table.data_ptr(), block_table.shape[1],
                                   cache_seqlens.data_ptr(), float(sm_scale), int(bool(is_causal)), int(is_fp8),
                                   kv_scales.data_ptr() if kv_scales is not None else None, ws.data_ptr(),
                                   ws.nbytes, o.data_ptr(), z.data_ptr())
        _check(lib().mla_shared_prefix_decode(ctypes.byref(a), handle))
        return o, z

    return _launch(dev, stream, call)


def index_topk_workspace_size(num_tokens: int, block_table_stride: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().mla_index_topk_workspace_size(num_tokens, block_table_stride, ctypes.byref(n)))
    return n.value


def index_topk(q_codes: torch.Tensor, q_scales: torch.Tensor, weights: torch.Tensor, row_offsets: torch.Tensor,
               k_codes: torch.Tensor, k_scales: torch.Tensor, block_table: torch.Tensor, cache_seqlens: torch.Tensor,
               topk: int, relu: bool = False, max_new_tokens: Optional[int] = None,
               indices: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """FP8 top-k indexer (mla_index_topk).  q_codes uint8 [T, h_idx, 128] (E4M3 codes), q_scales and
    weights fp32 [T, h_idx], row_offsets int32 [batch + 1], k_codes uint8 [num_pages, 64, 128],
    k_scales fp32 [num_pages, 64], block_table int32 [batch, stride], cache_seqlens int32 [batch].
    Returns int32 [T, topk] key ids (descending score, -1 fill).  Without max_new_tokens the
    largest row count is read from row_offsets (one device-to-host copy)."""
    if not torch.is_tensor(q_codes) or q_codes.device.type != "cuda":
        raise ValueError("q_codes must be a CUDA tensor")
    dev = q_codes.device
    _need(q_codes, "q_codes", torch.uint8, dev, 3)
    T, h_idx, d = q_codes.shape
    if d != 128:
        raise ValueError(f"q_codes must be [num_tokens, h_idx, 128] (got {tuple(q_codes.shape)})")
    _need(q_scales, "q_scales", torch.float32, dev, 2)
    _need(weights, "weights", torch.float32, dev, 2)
    if tuple(q_scales.shape) != (T, h_idx) or tuple(weights.shape) != (T, h_idx):
        raise ValueError("q_scales and weights must be [num_tokens, h_idx]")
    _need(row_offsets, "row_offsets", torch.int32, dev, 1)
    _need(k_codes, "k_codes", torch.uint8, dev, 3)
    if k_codes.shape[2] != 128:
        raise ValueError(f"k_codes must be [num_pages, page_size, 128] (got {tuple(k_codes.shape)})")
    _need(k_scales, "k_scales", torch.float32, dev, 2)
    if tuple(k_scales.shape) != tuple(k_codes.shape[:2]):
        raise ValueError("k_scales must be [num_pages, page_size]")
    _need(block_table, "block_table", torch.int32, dev, 2)
    _need(cache_seqlens, "cache_seqlens", torch.int32, dev, 1)
    batch = cache_seqlens.shape[0]
    if row_offsets.shape[0] != batch + 1 or block_table.shape[0] != batch:
        raise ValueError("row_offsets must have batch + 1 entries and block_table batch rows")
    if max_new_tokens is None:
        max_new_tokens = max(1, int(torch.diff(row_offsets).max().item())) if batch > 0 else 1
    if indices is None:
        indices = torch.empty((T, topk), dtype=torch.int32, device=dev)
    _need(indices, "indices", torch.int32, dev)
    if indices.numel() != T * topk:
        raise ValueError("indices has the wrong size")
    if workspace is None:
        workspace = torch.empty(max(16, index_topk_workspace_size(T, block_table.shape[1])), dtype=torch.uint8,
                                device=dev)
    a = IndexTopkArgs()
    a.q_codes, a.q_scales, a.weights = q_codes.data_ptr(), q_scales.data_ptr(), weights.data_ptr()
    a.num_tokens, a.h_idx = T, h_idx
    a.row_offsets, a.batch, a.max_new_tokens = row_offsets.data_ptr(), batch, int(max_new_tokens)
    a.k_codes, a.k_scales = k_codes.data_ptr(), k_scales.data_ptr()
    a.num_pages, a.page_size = k_codes.shape[0], k_codes.shape[1]
    a.block_table, a.block_table_stride = block_table.data_ptr(), block_table.shape[1]
    a.cache_seqlens = cache_seqlens.data_ptr()
    a.relu, a.topk = int(bool(relu)), int(topk)
    a.workspace = workspace.data_ptr()
    a.workspace_bytes = workspace.numel() * workspace.element_size()
    a.indices = indices.data_ptr()
    _check(lib().mla_index_topk(ctypes.byref(a), _stream(stream)))
    return indices.view(T, topk)


def device_status(stream=None, raise_on_error: bool = False) -> int:
    """Synchronise the stream, return and clear the device status bits."""
    flags = ctypes.c_uint32()
    st = lib().mla_get_device_status(_stream(stream), ctypes.byref(flags))
    if raise_on_error:
        _check(st)
    elif st not in (MLA_OK, 5, 6, 1):
        _check(st)
    return flags.value


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libmla.so for sm_103a (nvcc) into the package's _build folder."""
    global _lib
    path = _build.build(force=force, verbose=verbose)
    return path
