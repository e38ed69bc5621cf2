"""The paged-cache operators together, as a serving loop runs them: pages for the new tokens, their rows
into the cache, then attention over what is cached, step after step, against a 64-bit reference that
keeps every token's values in plain lists."""
import numpy as np
import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from paged_reference import attend, check, i32

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5
PAGE = 64


def stored_values(x, fmt):
    """The float64 values that rows written from bf16 [n, 576] stand for."""
    if fmt == "bf16":
        return x.double()
    t = x[:, :512].float().reshape(len(x), 4 if fmt == "fp8" else 1, -1)
    amax = t.abs().amax(-1, keepdim=True)
    # (a tensor divisor: torch divides by a Python number through its reciprocal, an ulp off)
    s = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    lat = ((t / s).to(torch.float8_e4m3fn).float() * s).to(torch.bfloat16).double().reshape(len(x), 512)
    return torch.cat([lat, x[:, 512:].double()], 1)


def empty_cache(pages, fmt):
    if fmt == "bf16":
        return torch.full((pages, PAGE, 1, 576), float("nan"), dtype=torch.bfloat16, device="cuda"), None
    row = 656 if fmt == "fp8" else 640
    kv = torch.full((pages, PAGE, 1, row), 0xFF, dtype=torch.uint8, device="cuda")
    return kv, torch.full((pages, PAGE), float("nan"), device="cuda") if fmt == "fp8_token" else None


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("h_q", [16, 128])
def test_prefill_then_decode_steps(fmt, h_q):
    rng = np.random.default_rng(1)
    g = torch.Generator("cuda").manual_seed(1)
    batch, pages, prefix, window, sinks = 5, 90, 200, 150, 4
    kv, sc = empty_cache(pages, fmt)
    free = i32(rng.permutation(pages))
    cursor = i32([0])
    # the shared prefix is a request of its own
    ptab = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    px = torch.randn(prefix, 576, generator=g, device="cuda").to(torch.bfloat16)
    plen, _, slots, cursor = mla.assign_pages(i32([0]), i32([prefix]), free, cursor, ptab, prefix, num_pages=pages)
    mla.cache_store(px[:, :512], px[:, 512:], slots, kv, kv_scales=sc)
    shared = stored_values(px, fmt)

    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    table = torch.full((batch, 9), -1, dtype=torch.int32, device="cuda")
    tokens = [torch.zeros(0, 576, dtype=torch.float64, device="cuda") for _ in range(batch)]
    for step in range(6):
        # a ragged prefill, then two query tokens per request (a step may hold none for a request)
        new = rng.integers(1, 330, batch) if step == 0 else np.full(batch, 2)
        pad = step % 3
        n = int(new.sum()) + pad
        x = torch.randn(n, 640, generator=g, device="cuda").to(torch.bfloat16)[:, 64:]  # a slice of wider rows
        lens, offsets, slots, cursor = mla.assign_pages(lens, i32(new), free, cursor, table, n, num_pages=pages,
                                                        cache_seqlens=lens, next_cursor=cursor)
        mla.cache_store(x[:, :512], x[:, 512:], slots, kv, kv_scales=sc)
        at = offsets.tolist()
        for b in range(batch):
            tokens[b] = torch.cat([tokens[b], stored_values(x[at[b]:at[b + 1]], fmt)])
        assert lens.tolist() == [len(t) for t in tokens]
        if step == 0:
            continue
        q = torch.randn(batch, 2, h_q, 576, generator=g, device="cuda").to(torch.bfloat16)
        got_w = mla.window_decode(q, kv, table, lens, SCALE, window=window, sinks=sinks, kv_scales=sc)
        got_p = mla.shared_prefix_decode(q, kv, ptab[0], plen, table, lens, SCALE, is_causal=True, kv_scales=sc)
        sched, ns = mla.get_metadata(lens, h_q=h_q, s_q=2, topk=0, is_fp8=fmt != "bf16")
        got_d = mla.decode(q, kv, table, lens, SCALE, sched, ns, is_causal=True, kv_scales=sc)
        assert mla.device_status() == 0
        want = {"w": [], "p": [], "d": []}
        for b in range(batch):
            for i in range(2):
                last = len(tokens[b]) - 2 + i
                own = tokens[b][:last + 1]
                sees = [t for t in range(last + 1) if t < sinks or t > last - window]
                want["w"].append(attend(q[b, i], own[torch.tensor(sees, device="cuda")], SCALE))
                want["p"].append(attend(q[b, i], torch.cat([shared, own]), SCALE))
                want["d"].append(attend(q[b, i], own, SCALE))
        for k, got in (("w", got_w), ("p", got_p), ("d", got_d)):
            ref = tuple(torch.stack([w[j] for w in want[k]]).view(batch, 2, h_q, *([512] if j != 1 else []))
                        for j in range(3))
            check(*got, ref, f"{fmt} step {step} {k}")


def test_a_decode_step_as_one_graph():
    # pages, store and windowed attention recorded once and replayed: every replay appends a token
    g = torch.Generator("cuda").manual_seed(3)
    batch, pages, h_q, window, sinks = 3, 40, 16, 70, 2
    kv, _ = empty_cache(pages, "fp8")
    free, cursor = i32(np.random.default_rng(2).permutation(pages)), i32([0])
    lens, new = i32([0] * batch), i32([1] * batch)
    table = torch.full((batch, 6), -1, dtype=torch.int32, device="cuda")
    x = torch.zeros(batch, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(batch, 1, h_q, 576, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.assign_pages(lens, new, free, cursor, table, batch, num_pages=pages, cache_seqlens=lens, next_cursor=cursor,
                         slot_map=(slots := torch.empty(batch, dtype=torch.int32, device="cuda")))
        mla.cache_store(x[:, :512], x[:, 512:], slots, kv)
        out, lse = mla.window_decode(q, kv, table, lens, SCALE, window=window, sinks=sinks)
    tokens = [[] for _ in range(batch)]
    for step in range(150):
        x.copy_(torch.randn(batch, 576, generator=g, device="cuda"))
        q.copy_(torch.randn(batch, 1, h_q, 576, generator=g, device="cuda"))
        graph.replay()
        v = stored_values(x, "fp8")
        for b in range(batch):
            tokens[b].append(v[b])
        if step % 10 == 9 or step in (0, 63, 64, 65):
            n = len(tokens[0])
            sees = [t for t in range(n) if t < sinks or t > n - 1 - window]
            ref = [attend(q[b, 0], torch.stack([tokens[b][t] for t in sees]), SCALE) for b in range(batch)]
            ref = tuple(torch.stack([r[j] for r in ref]).view(batch, 1, h_q, *([512] if j != 1 else [])) for j in range(3))
            check(out, lse, ref, f"step {step}")
    assert lens.tolist() == [150] * batch
    assert mla.device_status() == 0
