"""The FP4 cache and prompt attention together, as serving runs them: a prompt comes in chunks (pages, store, the
context read back and projected up, attention over it), then tokens one by one (pages, store, windowed decode), in
every row format, against a 64-bit reference that keeps every token's stored values in plain lists."""
import numpy as np
import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from fp4_reference import ROW, stored
from paged_reference import attend, check, i32
from test_gpu_paged_step import empty_cache, stored_values
from test_gpu_prompt import reference

pytestmark = pytest.mark.gpu
PAGE = 64
D_SCALE, P_SCALE = 576 ** -0.5, 192 ** -0.5


def make_cache(pages, fmt):
    if fmt != "fp4":
        return empty_cache(pages, fmt)
    return torch.full((pages, PAGE, 1, ROW), 0xFF, dtype=torch.uint8, device="cuda"), None


@pytest.mark.parametrize("fmt", ["fp4", "bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("heads", [16, 40])
def test_chunked_prefill_then_decode(fmt, heads):
    rng = np.random.default_rng(5)
    g = torch.Generator("cuda").manual_seed(5)
    batch, pages = 4, 80
    kv, sc = make_cache(pages, fmt)
    values = stored if fmt == "fp4" else lambda x: stored_values(x, fmt)
    w_up = (torch.randn(512, heads * 256, generator=g, device="cuda") * 512 ** -0.5).to(torch.bfloat16)
    free, cursor = i32(rng.permutation(pages)), i32([0])
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    table = torch.full((batch, 16), -1, dtype=torch.int32, device="cuda")
    tokens = [torch.zeros(0, 576, dtype=torch.float64, device="cuda") for _ in range(batch)]

    def append(new, pad):
        nonlocal lens, cursor
        n = int(sum(new)) + pad
        x = torch.randn(n, 640, generator=g, device="cuda").to(torch.bfloat16)[:, 64:]  # a slice of wider rows
        lens, offsets, slots, cursor = mla.assign_pages(lens, i32(new), free, cursor, table, n, num_pages=pages,
                                                        cache_seqlens=lens, next_cursor=cursor)
        mla.cache_store(x[:, :512], x[:, 512:], slots, kv, kv_scales=sc)
        at = offsets.tolist()
        for b in range(batch):
            if at[b + 1] > at[b]:
                tokens[b] = torch.cat([tokens[b], values(x[at[b]:at[b + 1]])])
        return offsets, n

    for step in range(3):
        new = [[300, 5, 64, 129], [77, 0, 200, 1], [1, 333, 0, 60]][step]
        q_offsets, n = append(new, pad=step)
        k_offsets = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), lens.cumsum(0).int()])
        total = sum(len(t) for t in tokens)
        rows = mla.cache_load(kv, table, k_offsets, total, kv_scales=sc)
        assert torch.equal(rows.double(), torch.cat(tokens))
        up = (rows[:, :512] @ w_up).view(total, heads, 256)
        q = torch.randn(n, heads, 192, generator=g, device="cuda").to(torch.bfloat16)
        args = (q, up[..., :128], rows[:, 512:], up[..., 128:], q_offsets, k_offsets)
        out, lse = mla.prompt_attention(*args, P_SCALE)
        assert mla.device_status() == 0
        real = int(sum(new))
        check(out[:real], lse[:real], tuple(w[:real] for w in reference(*args)), f"chunk {step}")

    for step in range(4):
        append([1] * batch, pad=0)
        q = torch.randn(batch, 1, heads, 576, generator=g, device="cuda").to(torch.bfloat16)
        for window, sinks in ((1 << 30, 0), (100, 4)):
            got = mla.window_decode(q, kv, table, lens, D_SCALE, window=window, sinks=sinks, kv_scales=sc)
            want = []
            for b in range(batch):
                last = len(tokens[b]) - 1
                sees = [t for t in range(last + 1) if t < sinks or t > last - window]
                want.append(attend(q[b, 0], tokens[b][torch.tensor(sees, device="cuda")], D_SCALE))
            want = tuple(torch.stack([w[j] for w in want]).view(batch, 1, heads, *([512] if j != 1 else [])) for j in range(3))
            check(*got, want, f"{fmt if fmt != 'bf16' else ''} step {step} window {window}")
    assert mla.device_status() == 0


def test_a_decode_step_over_fp4_as_one_graph():
    g = torch.Generator("cuda").manual_seed(3)
    batch, pages, h_q, window, sinks = 3, 40, 16, 70, 2
    kv, _ = make_cache(pages, "fp4")
    free, cursor = i32(np.random.default_rng(2).permutation(pages)), i32([0])
    lens, new = i32([0] * batch), i32([1] * batch)
    table = torch.full((batch, 6), -1, dtype=torch.int32, device="cuda")
    x = torch.zeros(batch, 576, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(batch, 1, h_q, 576, dtype=torch.bfloat16, device="cuda")
    row_offsets = i32(range(batch + 1))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.assign_pages(lens, new, free, cursor, table, batch, num_pages=pages, cache_seqlens=lens, next_cursor=cursor,
                         slot_map=(slots := torch.empty(batch, dtype=torch.int32, device="cuda")))
        mla.cache_store(x[:, :512], x[:, 512:], slots, kv)
        back = mla.cache_load(kv, table, row_offsets, batch)  # each request's first token
        out, lse = mla.window_decode(q, kv, table, lens, D_SCALE, window=window, sinks=sinks)
    tokens = [[] for _ in range(batch)]
    for step in range(150):
        x.copy_(torch.randn(batch, 576, generator=g, device="cuda"))
        q.copy_(torch.randn(batch, 1, h_q, 576, generator=g, device="cuda"))
        graph.replay()
        v = stored(x)
        for b in range(batch):
            tokens[b].append(v[b])
        if step % 10 == 9 or step in (0, 63, 64, 65):
            n = len(tokens[0])
            sees = [t for t in range(n) if t < sinks or t > n - 1 - window]
            ref = [attend(q[b, 0], torch.stack([tokens[b][t] for t in sees]), D_SCALE) for b in range(batch)]
            ref = tuple(torch.stack([r[j] for r in ref]).view(batch, 1, h_q, *([512] if j != 1 else [])) for j in range(3))
            check(out, lse, ref, f"step {step}")
            assert torch.equal(back.double(), torch.stack([tokens[b][0] for b in range(batch)]))
    assert lens.tolist() == [150] * batch
    assert mla.device_status() == 0
