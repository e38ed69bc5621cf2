"""What a call of the FP4 decode and of prompt attention asks of the CUDA runtime beside its launches."""
import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from paged_reference import i32

pytestmark = pytest.mark.gpu


def runtime_calls(call, n=4):
    """Names of the runtime's functions in n calls, after two that are not counted."""
    call()
    call()
    torch.cuda.synchronize()
    activities = [torch.profiler.ProfilerActivity.CPU, torch.profiler.ProfilerActivity.CUDA]
    with torch.profiler.profile(activities=activities):  # (the first of a process may miss calls)
        call()
        torch.cuda.synchronize()
    with torch.profiler.profile(activities=activities) as prof:
        for _ in range(n):
            call()
        torch.cuda.synchronize()
    return [e.name for e in prof.events() if e.name.startswith("cuda") or e.name.startswith("cuLaunch")]


def checked(names, launches):
    if not any("Launch" in n for n in names):
        pytest.skip("the profiler records no runtime calls here")
    assert sum("Launch" in n for n in names) == launches, names
    assert not [n for n in names if n.startswith("cudaFunc")], names


@pytest.mark.parametrize("h_q", [16, 128])
def test_fp4_decode_asks_for_no_attributes(h_q):
    q = torch.zeros(1, 1, h_q, 576, device="cuda", dtype=torch.bfloat16)
    kv = torch.zeros(2, 64, 1, 400, device="cuda", dtype=torch.uint8)
    table, lens = i32([[0, 1]]), i32([100])
    names = runtime_calls(lambda: mla.window_decode(q, kv, table, lens, 0.1, window=64))
    checked(names, 4)  # (a cluster: one launch a call)


@pytest.mark.parametrize("heads,launches", [(2, 4), (200, 8)])  # (items found by the CTAs; behind a plan)
def test_prompt_attention_asks_for_no_attributes(heads, launches):
    q = torch.zeros(10, heads, 192, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(10, heads, 128, device="cuda", dtype=torch.bfloat16)
    rope = torch.zeros(10, 64, device="cuda", dtype=torch.bfloat16)
    off = i32([0, 10])
    checked(runtime_calls(lambda: mla.prompt_attention(q, k, rope, k, off, off, 0.1)), launches)


@pytest.mark.parametrize("batch,h_q,keys,window,launches", [
    (100, 16, 600, 512, 1), (4, 16, 2100, 2048, 1), (30, 128, 1100, 1024, 1),  # on clusters
    (16, 16, 4200, 4096, 2), (2, 256, 4200, 4096, 2), (200, 16, 600, 512, 2), (32, 16, 8191, 1 << 30, 2),
    (100, 16, 8191, 1 << 30, 2), (38, 128, 16384, 1 << 30, 2)])  # a schedule and a merge
def test_fp4_decode_takes_the_side_that_was_measured_faster(batch, h_q, keys, window, launches):
    pages = -(-keys // 64)
    q = torch.zeros(batch, 1, h_q, 576, device="cuda", dtype=torch.bfloat16)
    kv = torch.zeros(pages, 64, 1, 400, device="cuda", dtype=torch.uint8)
    table, lens = torch.arange(pages, device="cuda", dtype=torch.int32).repeat(batch, 1), i32([keys] * batch)
    names = runtime_calls(lambda: mla.window_decode(q, kv, table, lens, 0.1, window=window))
    checked(names, 4 * launches)
