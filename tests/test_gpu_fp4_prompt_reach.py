"""The FP4 cache, cache reads and prompt attention at the ends of their documented ranges: caches and batches past
4 GiB, tensors whose strides run the other way, calls without tokens, calls from several host threads at once."""
import threading

import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from fp4_reference import ROW, quantise, rows_of, stored
from paged_reference import ROW as ROWS
from paged_reference import attend, check, i32
from test_gpu_prompt import SCALE, compare, inputs, reference

pytestmark = pytest.mark.gpu
PAGE = 64


def test_fp4_rows_past_4_gib():
    pages = (5 << 30) // (PAGE * ROW)
    kv = torch.empty(pages, PAGE, 1, ROW, dtype=torch.uint8, device="cuda")
    n = 700
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(n, 576, generator=g, device="cuda").to(torch.bfloat16)
    ids = [pages - 1 - 7 * i for i in range(-(-n // PAGE))]
    assert min(ids) * PAGE * ROW > 2 ** 32
    at = torch.arange(n, device="cuda")
    slots = torch.tensor(ids, device="cuda")[at // PAGE] * PAGE + at % PAGE
    kv.view(-1, ROW)[:2 * PAGE] = 0xFF  # (where offsets of 32 bits would be found)
    kv.view(-1, ROW)[pages - 7 * len(ids):] = 0xFF
    mla.cache_store(x[:, :512], x[:, 512:], slots.int(), kv)
    assert torch.equal(kv.view(-1, ROW)[slots], rows_of(*quantise(x[:, :512]), x[:, 512:]))
    rows = mla.cache_load(kv, i32([ids]), i32([0, n]), n)
    assert torch.equal(rows.double(), stored(x))
    for h_q in (16, 128):
        q = torch.randn(1, 1, h_q, 576, generator=g, device="cuda").to(torch.bfloat16)
        out, lse = mla.window_decode(q, kv, i32([ids]), i32([n]), 576 ** -0.5, window=1 << 30)
        want = attend(q[0, 0], stored(x), 576 ** -0.5)
        check(out, lse, tuple(w[None, None] for w in want), f"{h_q} heads")
    assert mla.device_status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_token"])
def test_reads_past_4_gib(fmt):
    pages = (5 << 30) // (PAGE * ROWS[fmt])
    raw = torch.empty(pages * PAGE, ROWS[fmt], dtype=torch.uint8, device="cuda")
    raw[-3 * PAGE:] = torch.randint(0, 100, (3 * PAGE, ROWS[fmt]), device="cuda", dtype=torch.uint8)
    raw[:3 * PAGE] = 0
    kv = raw.view(pages, PAGE, 1, -1)
    scales = torch.ones(pages, PAGE, device="cuda") if fmt == "fp8_token" else None
    small = raw[-3 * PAGE:].clone().view(3, PAGE, 1, -1)
    if fmt == "bf16":
        kv, small = kv.view(torch.bfloat16), small.view(torch.bfloat16)
    got = mla.cache_load(kv, i32([[pages - 1, pages - 3]]), i32([0, 100]), 100, kv_scales=scales)
    want = mla.cache_load(small, i32([[2, 0]]), i32([0, 100]), 100, kv_scales=None if scales is None else scales[:3].contiguous())
    assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and (want != 0).any()
    assert mla.device_status() == 0


def test_prompt_rows_past_4_gib():
    heads, many = 128, 140000  # q 6.9 GB, out 4.6 GB, the last sequence behind all of it
    q, k_nope, k_rope, v, _, _ = inputs(heads, heads, [(200, 300)], seed=2)
    big = torch.zeros(many + 200, heads, 192, device="cuda", dtype=torch.bfloat16)
    big[many:] = q
    out, lse = mla.prompt_attention(big, k_nope, k_rope, v, i32([0, many, many + 200]), i32([0, 0, 300]), SCALE)
    assert mla.device_status() == 0
    assert (out[:many] == 0).all() and (lse[:many] == -float("inf")).all()
    check(out[many:], lse[many:], reference(q, k_nope, k_rope, v, i32([0, 200]), i32([0, 300])), "the last sequence")


@pytest.mark.parametrize("lens", [[(300, 700), (5, 5)], [(9, 4000)]])
@pytest.mark.parametrize("h_q,h_kv", [(4, 2), (3, 1)])
def test_heads_that_lie_before_rows(lens, h_q, h_kv):
    # [heads, rows, values] in memory: the stride of a head is the longer one
    q, k_nope, k_rope, v, qo, ko = inputs(h_q, h_kv, lens, seed=5)

    def turned(t):
        return t.transpose(0, 1).contiguous().transpose(0, 1)

    args = turned(q), turned(k_nope), k_rope, turned(v), qo, ko
    assert args[0].stride(1) > args[0].stride(0)
    compare(args, "heads first")
    want = mla.prompt_attention(q, k_nope, k_rope, v, qo, ko, SCALE)
    got = mla.prompt_attention(*args, SCALE)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_calls_without_tokens():
    kv = torch.full((2, PAGE, 1, ROW), 7, dtype=torch.uint8, device="cuda")
    none = torch.empty(0, 576, device="cuda", dtype=torch.bfloat16)
    mla.cache_store(none[:, :512], none[:, 512:], i32([]), kv)
    assert (kv == 7).all()
    assert mla.cache_load(kv, i32([[0], [1]]), i32([0, 0, 0]), 0).shape == (0, 576)
    out = torch.full((3, 576), 5.0, device="cuda", dtype=torch.bfloat16)
    mla.cache_load(kv, i32([[0], [1]]), i32([0, 0, 0]), 3, out=out)
    assert (out == 5).all()
    q = torch.ones(2, 3, 16, 576, device="cuda", dtype=torch.bfloat16)
    out, lse = mla.window_decode(q, kv, i32([[-1], [-1]]), i32([0, 0]), 0.1, window=1)
    assert (out == 0).all() and (lse == -float("inf")).all()
    assert mla.device_status() == 0


def test_host_threads_at_once():
    # each thread its own stream, workspaces and sizes: planned prompts, shared-out ones, FP4 decode of 16 and 32 rows a CTA
    jobs = []
    for i, (heads, lens) in enumerate([(16, [(300, 400)] * 8), (2, [(5, 6000)]), (40, [(129, 129)] * 3)]):
        args = inputs(heads, heads, lens, seed=i)
        jobs.append(lambda a=args: mla.prompt_attention(*a, SCALE))
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(64 * PAGE, 576, generator=g, device="cuda").to(torch.bfloat16)
    kv = torch.zeros(64, PAGE, 1, ROW, dtype=torch.uint8, device="cuda")
    mla.cache_store(x[:, :512], x[:, 512:], torch.arange(64 * PAGE, device="cuda", dtype=torch.int32), kv)
    table = torch.arange(64, device="cuda", dtype=torch.int32).view(4, 16).contiguous()
    for h_q, window in ((16, 1 << 30), (128, 200)):
        q = torch.randn(4, 1, h_q, 576, generator=g, device="cuda").to(torch.bfloat16)
        lens = i32([1024, 1000, 3, 517])
        jobs.append(lambda q=q, lens=lens, w=window: mla.window_decode(q, kv, table, lens, 576 ** -0.5, window=w))
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(40):
                out, lse = jobs[i]()
                torch.cuda.current_stream().synchronize()
                if not (torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert mla.device_status() == 0
