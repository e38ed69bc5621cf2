"""Argument structs and refusals of the paged-cache operators (no GPU: invalid calls return before
any device is touched)."""
import ctypes
import os
import re

import pytest
import torch

import paged_mla_decode_07_gb300 as mla

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mla.h")
P = 1 << 20  # a plausible device address, never dereferenced


@pytest.fixture(scope="module")
def lib():
    mla.build()
    return mla.lib()


STRUCTS = [("mla_assign_pages_args", mla.AssignPagesArgs), ("mla_cache_store_args", mla.CacheStoreArgs),
           ("mla_window_decode_args", mla.WindowDecodeArgs),
           ("mla_shared_prefix_decode_args", mla.SharedPrefixDecodeArgs)]
CTYPES = {"int": ctypes.c_int, "int64_t": ctypes.c_int64, "float": ctypes.c_float, "size_t": ctypes.c_size_t}


@pytest.mark.parametrize("struct,cls", STRUCTS)
def test_structs_match_the_header(struct, cls):
    text = open(HEADER).read()
    body = re.search(r"typedef struct \{((?:(?!typedef struct).)*?)\} " + struct + ";", text, flags=re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        kind, names = re.match(r"(?:const\s+)?(\w+)\s*(.*)", decl, flags=re.S).groups()
        for n in names.split(","):
            n = n.strip()
            fields.append((n.lstrip("*").strip(), ctypes.c_void_p if n.startswith("*") else CTYPES[kind]))
    assert fields == list(cls._fields_)


def make(cls, base, **kw):
    a = cls()
    for f, v in {**base, **kw}.items():
        setattr(a, f, v)
    return ctypes.byref(a)


PAGES = dict(cache_lengths=P, new_tokens=2 * P, batch=2, free_pages=3 * P, num_free=4, free_cursor=4 * P, block_table=5 * P,
             block_table_stride=3, num_pages=100, num_tokens=5, cache_seqlens=6 * P, row_offsets=7 * P, slot_map=8 * P,
             next_cursor=9 * P)
STORE = dict(latent=P, latent_stride=512, rope=2 * P, rope_stride=64, slot_map=3 * P, num_tokens=3, kvcache=4 * P,
             num_pages=2, page_size=64, is_fp8=1, kv_scales=None)
WINDOW = dict(q=P, batch=1, s_q=1, h_q=16, kvcache=2 * P, num_pages=2, page_size=64, block_table=3 * P,
              block_table_stride=2, cache_seqlens=4 * P, sm_scale=0.1, window=5, sinks=0, is_fp8=0, kv_scales=None,
              workspace=5 * P, workspace_bytes=1 << 40, out=6 * P, lse=7 * P)
PREFIX = {k: v for k, v in WINDOW.items() if k not in ("window", "sinks")} | dict(
    prefix_table=8 * P, prefix_table_len=4, prefix_length=9 * P, is_causal=1)


@pytest.mark.parametrize("field,value,status,needle", [
    ("batch", 0, 1, "batch"), ("batch", 16385, 2, "batch"), ("cache_lengths", None, 1, "cache_lengths is NULL"),
    ("new_tokens", P + 2, 1, "new_tokens is not 4-byte aligned"), ("free_pages", None, 1, "free_pages is NULL"),
    ("num_free", -1, 1, "num_free"), ("num_tokens", -1, 1, "num_tokens"), ("num_pages", 0, 1, "num_pages"),
    ("num_pages", 2 ** 25, 2, "num_pages"), ("block_table_stride", 0, 1, "block_table_stride"),
    ("slot_map", None, 1, "slot_map is NULL"), ("next_cursor", None, 1, "next_cursor is NULL"),
    ("cache_seqlens", P + 4, 1, "cache_seqlens overlaps cache_lengths"),
    ("cache_seqlens", 2 * P, 1, "cache_seqlens overlaps new_tokens"),
    ("next_cursor", 3 * P, 1, "next_cursor overlaps free_pages"),
    ("slot_map", 7 * P + 8, 1, "slot_map overlaps row_offsets"),
    ("block_table", P - 20, 1, "block_table overlaps cache_lengths")])
def test_assign_pages_refusals(lib, field, value, status, needle):
    assert lib.mla_assign_pages(make(mla.AssignPagesArgs, PAGES, **{field: value}), None) == status
    assert needle in mla.last_error()


@pytest.mark.parametrize("field,value,status,needle", [
    ("latent", None, 1, "latent is NULL"), ("rope", None, 1, "rope is NULL"), ("slot_map", None, 1, "slot_map is NULL"),
    ("kvcache", None, 1, "kvcache is NULL"), ("latent", P + 8, 1, "latent is not 16-byte aligned"),
    ("rope", P + 2, 1, "rope is not 16-byte aligned"), ("latent_stride", 516, 1, "latent_stride"),
    ("rope_stride", -64, 1, "rope_stride"), ("num_tokens", -1, 1, "num_tokens"), ("page_size", 16, 2, "page_size"),
    ("num_pages", 0, 1, "num_pages"), ("num_pages", 2 ** 25, 2, "num_pages"), ("is_fp8", 2, 1, "is_fp8")])
def test_cache_store_refusals(lib, field, value, status, needle):
    assert lib.mla_cache_store(make(mla.CacheStoreArgs, STORE, **{field: value}), None) == status
    assert needle in mla.last_error()
    assert lib.mla_cache_store(make(mla.CacheStoreArgs, STORE, is_fp8=0, kv_scales=P), None) == 1
    # no tokens: nothing to read, nothing launched
    assert lib.mla_cache_store(make(mla.CacheStoreArgs, STORE, num_tokens=0, latent=None, rope=None), None) == 0


COMMON = [("q", None, 1, "q is NULL"), ("kvcache", None, 1, "kvcache is NULL"), ("out", None, 1, "out is NULL"),
          ("lse", None, 1, "lse is NULL"), ("block_table", None, 1, "block_table is NULL"),
          ("cache_seqlens", None, 1, "cache_seqlens is NULL"), ("page_size", 128, 2, "page_size"),
          ("num_pages", 0, 1, "num_pages"), ("num_pages", 2 ** 25, 2, "num_pages"), ("q", P + 8, 1, "q is not"),
          ("kvcache", P + 8, 1, "kvcache is not"), ("out", P + 8, 1, "out is not"), ("sm_scale", float("inf"), 1, "sm_scale"),
          ("is_fp8", 7, 1, "is_fp8"), ("kv_scales", P, 1, "kv_scales given"), ("block_table_stride", 0, 1, "stride"),
          ("batch", 0, 1, "batch"), ("s_q", 0, 1, "s_q"), ("h_q", 0, 1, "h_q"), ("h_q", 1025, 2, "1024"),
          ("batch", 16385, 2, "16384"), ("block_table_stride", 2 ** 30, 2, "block table")]


@pytest.mark.parametrize("field,value,status,needle", COMMON + [("window", 0, 1, "window"), ("sinks", -1, 1, "sinks")])
def test_window_decode_refusals(lib, field, value, status, needle):
    assert lib.mla_window_decode(make(mla.WindowDecodeArgs, WINDOW, **{field: value}), None) == status
    assert needle in mla.last_error()


@pytest.mark.parametrize("field,value,status,needle", COMMON + [
    ("prefix_table", None, 1, "prefix_table is NULL"), ("prefix_length", None, 1, "prefix_length is NULL"),
    ("prefix_table_len", 0, 1, "prefix_table_len"), ("prefix_table_len", 2 ** 25, 2, "prefix_table_len")])
def test_shared_prefix_decode_refusals(lib, field, value, status, needle):
    assert lib.mla_shared_prefix_decode(make(mla.SharedPrefixDecodeArgs, PREFIX, **{field: value}), None) == status
    assert needle in mla.last_error()


def test_size_queries_refuse(lib):
    n = ctypes.c_size_t()
    assert lib.mla_window_decode_workspace_size(0, 16, 1, 0, ctypes.byref(n)) == 1
    assert lib.mla_window_decode_workspace_size(1, 16, 1, 0, None) == 1
    assert lib.mla_window_decode_workspace_size(1, 16, 1, 3, ctypes.byref(n)) == 1
    assert lib.mla_shared_prefix_decode_workspace_size(1, 16, 1, 0, 0, ctypes.byref(n)) == 1
    assert lib.mla_shared_prefix_decode_workspace_size(1, 2048, 1, 4, 0, ctypes.byref(n)) == 2
    assert lib.mla_assign_pages(None, None) == 1 and lib.mla_cache_store(None, None) == 1
    assert lib.mla_window_decode(None, None) == 1 and lib.mla_shared_prefix_decode(None, None) == 1


def test_binding_refuses_cpu_tensors():
    z = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="cache_lengths must be a CUDA tensor"):
        mla.assign_pages(z, z, z, z, z.view(1, 1), 1)
    with pytest.raises(ValueError, match="latent must be a CUDA tensor"):
        mla.cache_store(torch.zeros(1, 512), torch.zeros(1, 64), z, z)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        mla.window_decode(z, z, z, z, 1.0, window=1)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        mla.shared_prefix_decode(z, z, z, z, z, z, 1.0)
