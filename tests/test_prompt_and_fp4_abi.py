"""Argument structs and refusals of the FP4 cache, the cache read and prompt attention (no GPU: invalid
calls return before any device is touched)."""
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


STRUCTS = [("mla_fp4_cache_store_args", mla.Fp4CacheStoreArgs), ("mla_cache_load_args", mla.CacheLoadArgs),
           ("mla_fp4_decode_args", mla.Fp4DecodeArgs), ("mla_prompt_attention_args", mla.PromptAttentionArgs)]
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


STORE = dict(latent=P, latent_stride=512, rope=2 * P, rope_stride=64, slot_map=3 * P, num_tokens=3, kvcache=4 * P, num_pages=2,
             page_size=64)
LOAD = dict(kvcache=P, num_pages=2, page_size=64, format=3, kv_scales=None, block_table=2 * P, block_table_stride=2, batch=2,
            starts=None, row_offsets=3 * P, num_tokens=5, out=4 * P)
DECODE = dict(q=P, batch=1, s_q=1, h_q=16, kvcache=2 * P, num_pages=2, page_size=64, block_table=3 * P, block_table_stride=2,
              cache_seqlens=4 * P, sm_scale=0.1, window=5, sinks=0, workspace=5 * P, workspace_bytes=1 << 40, out=6 * P,
              lse=7 * P)
PROMPT = dict(q=P, q_stride=192 * 4, q_head_stride=192, num_q=9, h_q=4, k_nope=2 * P, k_nope_stride=256 * 2,
              k_nope_head_stride=256, k_rope=3 * P, k_rope_stride=576, v=4 * P, v_stride=256 * 2, v_head_stride=256, num_k=9,
              h_kv=2, q_offsets=5 * P, k_offsets=6 * P, batch=2, sm_scale=0.1, is_causal=1, workspace=7 * P,
              workspace_bytes=1 << 40, out=8 * P, lse=9 * P)


@pytest.mark.parametrize("field,value,status,needle", [
    ("latent", None, 1, "latent is NULL"), ("rope", None, 1, "rope is NULL"), ("slot_map", None, 1, "slot_map is NULL"),
    ("kvcache", None, 1, "kvcache is NULL"), ("latent", P + 8, 1, "latent is not"), ("kvcache", P + 8, 1, "kvcache is not"),
    ("latent_stride", 516, 1, "latent_stride"), ("rope_stride", -64, 1, "rope_stride"), ("num_tokens", -1, 1, "num_tokens"),
    ("page_size", 16, 2, "page_size"), ("num_pages", 0, 1, "num_pages"), ("num_pages", 2 ** 25, 2, "num_pages")])
def test_store_refusals(lib, field, value, status, needle):
    assert lib.mla_fp4_cache_store(make(mla.Fp4CacheStoreArgs, STORE, **{field: value}), None) == status
    assert needle in mla.last_error()
    assert lib.mla_fp4_cache_store(make(mla.Fp4CacheStoreArgs, STORE, num_tokens=0, latent=None, rope=None), None) == 0
    assert lib.mla_fp4_cache_store(None, None) == 1


@pytest.mark.parametrize("field,value,status,needle", [
    ("kvcache", None, 1, "kvcache is NULL"), ("block_table", None, 1, "block_table is NULL"),
    ("row_offsets", None, 1, "row_offsets is NULL"), ("out", None, 1, "out is NULL"), ("out", P + 8, 1, "out is not"),
    ("kvcache", P + 8, 1, "kvcache is not"), ("starts", P + 2, 1, "starts is not"), ("format", 4, 1, "format"),
    ("format", -1, 1, "format"), ("format", 2, 1, "kv_scales is NULL"), ("kv_scales", P, 1, "kv_scales given"),
    ("batch", 0, 1, "batch"), ("batch", 16385, 2, "batch"), ("page_size", 32, 2, "page_size"), ("num_pages", 0, 1, "num_pages"),
    ("num_pages", 2 ** 25, 2, "num_pages"), ("block_table_stride", 0, 1, "block_table_stride"),
    ("num_tokens", -1, 1, "num_tokens")])
def test_load_refusals(lib, field, value, status, needle):
    assert lib.mla_cache_load(make(mla.CacheLoadArgs, LOAD, **{field: value}), None) == status
    assert needle in mla.last_error()
    assert lib.mla_cache_load(make(mla.CacheLoadArgs, LOAD, num_tokens=0, out=None), None) == 0
    assert lib.mla_cache_load(None, None) == 1


@pytest.mark.parametrize("field,value,status,needle", [
    ("q", None, 1, "q is NULL"), ("kvcache", None, 1, "kvcache is NULL"), ("out", None, 1, "out is NULL"),
    ("lse", None, 1, "lse is NULL"), ("block_table", None, 1, "block_table is NULL"),
    ("cache_seqlens", None, 1, "cache_seqlens is NULL"), ("page_size", 128, 2, "page_size"), ("num_pages", 0, 1, "num_pages"),
    ("num_pages", 2 ** 25, 2, "num_pages"), ("q", P + 8, 1, "q is not"), ("kvcache", P + 8, 1, "kvcache is not"),
    ("out", P + 8, 1, "out is not"), ("sm_scale", float("nan"), 1, "sm_scale"), ("block_table_stride", 0, 1, "stride"),
    ("batch", 0, 1, "batch"), ("s_q", 0, 1, "s_q"), ("h_q", 0, 1, "h_q"), ("h_q", 1025, 2, "1024"),
    ("batch", 16385, 2, "16384"), ("block_table_stride", 2 ** 30, 2, "block table"), ("window", 0, 1, "window"),
    ("sinks", -1, 1, "sinks")])
def test_decode_refusals(lib, field, value, status, needle):
    assert lib.mla_fp4_decode(make(mla.Fp4DecodeArgs, DECODE, **{field: value}), None) == status
    assert needle in mla.last_error()
    assert lib.mla_fp4_decode(None, None) == 1


@pytest.mark.parametrize("field,value,status,needle", [
    ("q", None, 1, "q is NULL"), ("k_nope", None, 1, "k_nope is NULL"), ("k_rope", None, 1, "k_rope is NULL"),
    ("v", None, 1, "v is NULL"), ("q_offsets", None, 1, "q_offsets is NULL"), ("k_offsets", None, 1, "k_offsets is NULL"),
    ("out", None, 1, "out is NULL"), ("lse", None, 1, "lse is NULL"), ("q", P + 8, 1, "q is not"), ("v", P + 8, 1, "v is not"),
    ("k_rope", P + 2, 1, "k_rope is not"), ("out", P + 8, 1, "out is not"), ("q_stride", 770, 1, "q_stride"),
    ("q_head_stride", 0, 1, "q_head_stride"), ("k_nope_stride", -512, 1, "k_nope_stride"),
    ("v_head_stride", 100, 1, "v_head_stride"), ("k_rope_stride", 2 ** 40, 1, "k_rope_stride"), ("num_q", -1, 1, "num_q"),
    ("num_k", -1, 1, "num_k"), ("h_q", 0, 1, "h_q"), ("h_q", 3, 1, "multiple of h_kv"), ("h_kv", 0, 1, "multiple of h_kv"),
    ("h_q", 2048, 2, "1024"), ("batch", 0, 1, "batch"), ("batch", 16385, 2, "16384"), ("sm_scale", float("inf"), 1, "sm_scale")])
def test_prompt_refusals(lib, field, value, status, needle):
    assert lib.mla_prompt_attention(make(mla.PromptAttentionArgs, PROMPT, **{field: value}), None) == status
    assert needle in mla.last_error()


def test_prompt_sizes(lib):
    # rows x heads past 31 bits of blocks
    big = dict(num_q=2 ** 31 - 1, h_q=1024, q_head_stride=192)
    assert lib.mla_prompt_attention(make(mla.PromptAttentionArgs, PROMPT, **big), None) == 2
    assert "num_q" in mla.last_error()
    assert lib.mla_prompt_attention(None, None) == 1
    n = ctypes.c_size_t()
    for sizes, status in (((1000, 10, 2, 0), 1), ((-1, 10, 2, 1), 1), ((10, -1, 2, 1), 1), ((10, 10, 0, 1), 1), ((10, 10, 1025, 1), 2)):
        assert lib.mla_prompt_attention_workspace_size(*sizes, ctypes.byref(n)) == status
    assert lib.mla_prompt_attention_workspace_size(1000, 1000, 1, 1, None) == 1
    assert lib.mla_fp4_decode_workspace_size(0, 16, 1, ctypes.byref(n)) == 1
    assert lib.mla_fp4_decode_workspace_size(1, 16, 1, None) == 1


def test_binding_refuses_cpu_tensors():
    z = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="kvcache must be a CUDA tensor"):
        mla.cache_load(z, z, z, 1)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        mla.prompt_attention(z, z, z, z, z, z, 1.0)
