"""Windowed decode with sinks on the GPU against a 64-bit reference."""
import numpy as np
import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from gpu_helpers import Guarded, check_guards, overrides
from paged_reference import Cache, attend, check, i32, table

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5


def seen(L, s_q, i, window, sinks):
    last = L - s_q + i
    return [t for t in range(max(0, min(last + 1, L))) if t < sinks or t > last - window]


def problem(fmt, h_q, s_q, lens, window, sinks, seed=0, store_all=False, make=Cache):
    cache = make(fmt, seed, sum(-(-L // 64) for L in lens) + 3)
    g = torch.Generator("cuda").manual_seed(seed + 1)
    q = torch.randn(len(lens), s_q, h_q, 576, generator=g, device="cuda").to(torch.bfloat16)
    rows, want = [], []
    for b, L in enumerate(lens):
        sets = [seen(L, s_q, i, window, sinks) for i in range(s_q)]
        values, ids = cache.put(L, keep=None if store_all else set().union(*sets))
        rows.append(ids)
        for i in range(s_q):
            want.append(attend(q[b, i], values[torch.tensor(sets[i], dtype=torch.long, device="cuda")], SCALE))
    want = tuple(torch.stack([w[k] for w in want]).view(len(lens), s_q, h_q, *([512] if k != 1 else [])) for k in range(3))
    kv, sc = cache.tensors()
    return q, kv, sc, table(rows), i32(lens), want


def run(q, kv, sc, bt, lens, window, sinks, flags=0, **kw):
    b, s, h, _ = q.shape
    g_out, g_lse = Guarded(b * s * h * 1024), Guarded(b * s * h * 4)
    g_ws = Guarded(mla.window_decode_workspace_size(b, h_q=h, s_q=s, is_fp8=kv.dtype == torch.uint8))
    g_ws.body.fill_(0xFF)
    out, lse = mla.window_decode(q, kv, bt, lens, SCALE, window=window, sinks=sinks, kv_scales=sc,
                                 out=g_out.view(torch.bfloat16, (b, s, h, 512)),
                                 lse=g_lse.view(torch.float32, (b, s, h)), workspace=g_ws.body, **kw)
    assert mla.device_status() == flags
    check_guards({"out": g_out, "lse": g_lse, "workspace": g_ws}, "window_decode")
    return out, lse


LENS = (0, 1, 5, 63, 64, 65, 127, 128, 129, 300, 641, 1000)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 0), (64, 64), (100, 10), (130, 65), (256, 129),
                                          (1000, 0), (200, 5000), (2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("h_q,s_q", [(16, 1), (128, 1), (24, 3)])
def test_window_and_sinks(fmt, h_q, s_q, window, sinks):
    q, kv, sc, bt, lens, want = problem(fmt, h_q, s_q, LENS, window, sinks, seed=window % 1000 + sinks % 1000)
    check(*run(q, kv, sc, bt, lens, window, sinks), want, f"{fmt} {h_q}x{s_q} window {window} sinks {sinks}")


@pytest.mark.parametrize("h_q,s_q", [(1, 1), (8, 1), (8, 3), (20, 1), (32, 1), (33, 1), (64, 1), (16, 4), (65, 1), (40, 2),
                                     (128, 2), (96, 3), (100, 5), (1, 200), (512, 2)])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_row_counts(fmt, h_q, s_q):
    window, sinks = 150, 20
    q, kv, sc, bt, lens, want = problem(fmt, h_q, s_q, (0, 2, 64, 190, 777), window, sinks, seed=h_q * 7 + s_q)
    check(*run(q, kv, sc, bt, lens, window, sinks), want, f"{fmt} {h_q}x{s_q}")


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("h_q", [16, 128])
@pytest.mark.parametrize("parts", [1, 2, 7, 40, 300])
def test_forced_splits(fmt, h_q, parts):
    q, kv, sc, bt, lens, want = problem(fmt, h_q, 2, (0, 700, 64, 1500, 3), 400, 70, seed=parts)
    with overrides(num_parts=parts):
        got = run(q, kv, sc, bt, lens, 400, 70)
    check(*got, want, f"{fmt} {h_q} parts {parts}")


@pytest.mark.parametrize("fmt,h_q", [("bf16", 16), ("bf16", 128), ("fp8", 16), ("fp8_token", 128)])
@pytest.mark.parametrize("n,longest", [(330, 900), (255, 200), (256, 200), (257, 200), (2500, 100)])
def test_many_elements(fmt, h_q, n, longest):
    # several problems per thread of the schedule that every CTA makes
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, longest, n)]
    q, kv, sc, bt, L, want = problem(fmt, h_q, 1, lens, 200, 4, seed=5)
    check(*run(q, kv, sc, bt, L, 200, 4), want, f"{fmt} {h_q}")


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_a_window_over_everything_equals_dense_decode(fmt):
    lens = (700, 64, 1, 1300)
    q, kv, sc, bt, L, ref = problem(fmt, 16, 2, lens, 1 << 20, 0, seed=9)
    got = run(q, kv, sc, bt, L, 1 << 20, 0)
    sched, ns = mla.get_metadata(L, h_q=16, s_q=2, topk=0, is_fp8=fmt != "bf16")
    want = mla.decode(q, kv, bt, L, SCALE, sched, ns, is_causal=True)
    assert mla.device_status() == 0
    check(*got, ref, f"{fmt} windowed")
    check(*want, ref, f"{fmt} dense")


@pytest.mark.parametrize("fmt,h_q", [("bf16", 16), ("bf16", 128), ("fp8", 16), ("fp8", 128)])
def test_an_unusable_page_is_flagged_and_masked(fmt, h_q):
    lens, window, sinks = (900, 500), 300, 64
    q, kv, sc, bt, L, _ = problem(fmt, h_q, 1, lens, window, sinks, seed=4)
    lost = 900 // 64 - 1
    bt2 = bt.clone()
    bt2[0, lost] = kv.shape[0]
    got = run(q, kv, sc, bt2, L, window, sinks, flags=mla.DEVICE_BAD_PAGE)
    whole = run(q, kv, sc, bt, L, window, sinks)
    assert torch.isfinite(got[0]).all()
    # the other element is untouched; the masked keys lower the sum
    assert torch.allclose(got[1][1], whole[1][1], rtol=0, atol=2.0 ** -18)
    assert (got[1][0] < whole[1][0]).all()


def test_short_block_table_rows_are_flagged():
    q, kv, sc, bt, L, _ = problem("bf16", 16, 1, (900,), 300, 0, seed=4)
    run(q, kv, sc, bt[:, :14].contiguous(), L, 300, 0, flags=mla.DEVICE_BAD_PAGE)


def test_repeated_runs_and_graph_replays_agree():
    q, kv, sc, bt, L, want = problem("bf16", 128, 2, (900, 130, 64, 1700), 500, 30, seed=6, store_all=True)
    first = [t.clone() for t in run(q, kv, sc, bt, L, 500, 30)]
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    ws = torch.empty(mla.window_decode_workspace_size(4, h_q=128, s_q=2, is_fp8=False), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.window_decode(q, kv, bt, L, SCALE, window=500, sinks=30, out=out, lse=lse, workspace=ws)
    for _ in range(10):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    # the lengths are read when the graph runs
    L.fill_(64)
    graph.replay()
    again = run(q, kv, sc, bt, L, 500, 30)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_two_streams_with_their_own_workspaces():
    a = problem("bf16", 16, 1, (900, 130, 64, 1700), 500, 30, seed=6)
    b = problem("fp8", 64, 1, (300, 1200), 100, 3, seed=7)
    want = [run(*a[:5], 500, 30), run(*b[:5], 100, 3)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        got.append((mla.window_decode(a[0], a[1], a[3], a[4], SCALE, window=500, sinks=30, stream=streams[0]),
                    mla.window_decode(b[0], b[1], b[3], b[4], SCALE, window=100, sinks=3, stream=streams[1].cuda_stream)))
    torch.cuda.synchronize()
    assert mla.device_status() == 0
    for x, y in got:
        for g, w in ((x, want[0]), (y, want[1])):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


class FarScales(Cache):
    """FP8 keys whose scales lie six orders apart: small values, and among them tokens with all-zero
    tiles, which the format stores with the scale 1."""

    def rows(self, n):
        x = torch.randn(n, 512, generator=self.g, device="cuda") * 2.0 ** -20
        x[::5] = 0
        return self.encode(x, torch.randn(n, 64, generator=self.g, device="cuda"))

    def encode(self, x, rope):
        n = x.shape[0]
        rope = rope.to(torch.bfloat16)
        t = x.reshape(n, 4 if self.fmt == "fp8" else 1, -1)
        s = t.abs().amax(-1, keepdim=True) / torch.tensor(448.0, device="cuda")
        s = torch.where(s > 0, s, torch.ones_like(s))
        codes = (t / s).to(torch.float8_e4m3fn)
        lat = (codes.float() * s).to(torch.bfloat16).double().reshape(n, 512)
        parts = [codes.view(torch.uint8).reshape(n, 512)]
        if self.fmt == "fp8":
            parts.append(s.reshape(n, 4).contiguous().view(torch.uint8))
        parts.append(rope.contiguous().view(torch.uint8))
        return torch.cat([lat, rope.double()], 1), torch.cat(parts, 1), s.reshape(n) if self.fmt == "fp8_token" else None


class SmallCodes(FarScales):
    """FP8 keys whose codes are subnormal but for one per tile."""

    def rows(self, n):
        x = torch.randn(n, 512, generator=self.g, device="cuda").clamp(-3, 3) * 2.0 ** -9
        x[:, ::128] = 448.0
        return self.encode(x * 2.0 ** -10, torch.randn(n, 64, generator=self.g, device="cuda"))


@pytest.mark.parametrize("make", [FarScales, SmallCodes])
@pytest.mark.parametrize("fmt", ["fp8", "fp8_token"])
@pytest.mark.parametrize("h_q,s_q", [(8, 1), (16, 1), (20, 1), (64, 1), (128, 1), (24, 3)])
def test_scales_and_codes_far_apart(make, fmt, h_q, s_q):
    q, kv, sc, bt, lens, want = problem(fmt, h_q, s_q, (5, 64, 300, 777), 200, 20, seed=h_q, make=make)
    check(*run(q, kv, sc, bt, lens, 200, 20), want, f"{fmt} {h_q}x{s_q} {make.__name__}")


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("h_q,s_q", [(16, 1), (40, 1), (64, 2)])
@pytest.mark.parametrize("window,sinks", [(100, 0), (100, 70), (100, 2 ** 31 - 1), (2 ** 31 - 1, 5)])
def test_lengths_past_the_block_table(fmt, h_q, s_q, window, sinks):
    """The keys that the table has pages for are attended to at the positions that the length gives
    them; the missing ones are flagged, however many there are."""
    cache = Cache(fmt, h_q + sinks % 100, 3 * 4 + 3)
    lens = (2 ** 31 - 1, 2 ** 31 - 63, 192 + 1, 192 + 150)
    g = torch.Generator("cuda").manual_seed(h_q)
    q = torch.randn(len(lens), s_q, h_q, 576, generator=g, device="cuda").to(torch.bfloat16)
    rows, want = [], []
    reach = min(window, 1 << 30)
    for b, L in enumerate(lens):
        values, ids = cache.put(192)
        rows.append(ids)
        for i in range(s_q):
            last = L - s_q + i
            ids = [t for t in range(192) if t <= last and (t < sinks or t > last - reach)]
            want.append(attend(q[b, i], values[torch.tensor(ids, dtype=torch.long, device="cuda")], SCALE))
    want = tuple(torch.stack([w[k] for w in want]).view(len(lens), s_q, h_q, *([512] if k != 1 else [])) for k in range(3))
    kv, sc = cache.tensors()
    check(*run(q, kv, sc, table(rows), i32(lens), window, sinks, flags=mla.DEVICE_BAD_PAGE), want, f"{fmt} past the table")


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("h_q", [8, 40, 128])
@pytest.mark.parametrize("parts", [None, 40])
def test_a_seen_nan_is_not_lost(fmt, h_q, parts):
    """Whole problems and split ones alike: the element's rows and their lse are NaN, the others' are right."""
    lens = (700, 130, 300)
    q, kv, sc, bt, L, want = problem(fmt, h_q, 1, lens, 500, 10, seed=h_q, store_all=True)
    page, slot = int(bt[0, 650 // 64]), 650 % 64
    if fmt == "bf16":
        kv.view(torch.int16)[page, slot, 0, 77] = 0x7FC0
    else:
        kv[page, slot, 0, 512:516].view(torch.float32).fill_(float("nan"))
    if parts:
        with overrides(num_parts=parts):
            out, lse = run(q, kv, sc, bt, L, 500, 10)
    else:
        out, lse = run(q, kv, sc, bt, L, 500, 10)
    check(out[1:], lse[1:], tuple(w[1:] for w in want), f"{fmt} {h_q} beside NaN")
    assert torch.isnan(out[0]).any() and torch.isnan(lse[0]).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("n,h_q", [(1, 16), (3, 16), (9, 40), (17, 7), (30, 16), (50, 30), (70, 16), (75, 64), (140, 16), (152, 8)])
def test_batches_that_clusters_share(fmt, n, h_q):
    """Few and many short windows: every size of cluster, elements without keys and with a single page among them."""
    lens = [(37 * b * b + 11 * b) % 700 for b in range(n)]
    lens[n // 2] = 650
    q, kv, sc, bt, lens, want = problem(fmt, h_q, 1, lens, 300, 6, seed=n)
    got = run(q, kv, sc, bt, lens, 300, 6)
    check(*got, want, f"{fmt} {n} elements of {h_q} rows")
    again = run(q, kv, sc, bt, lens, 300, 6)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("fmt,h_q,n", [("bf16", 16, 4), ("fp8", 16, 4), ("fp8_token", 64, 3), ("bf16", 64, 40)])
def test_clusters_are_captured_and_follow_the_lengths(fmt, h_q, n):
    lens = [300 + 17 * b for b in range(n)]
    q, kv, sc, bt, L, want = problem(fmt, h_q, 1, lens, 200, 3, seed=n, store_all=True)
    out = torch.empty(n, 1, h_q, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(n, 1, h_q, device="cuda")
    ws = torch.empty(mla.window_decode_workspace_size(n, h_q=h_q, s_q=1, is_fp8=fmt != "bf16"), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.window_decode(q, kv, bt, L, SCALE, window=200, sinks=3, kv_scales=sc, out=out, lse=lse, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    check(out, lse, want, f"{fmt} replayed")
    for length in (0, 1, 64, 250):
        L.fill_(length)
        graph.replay()
        again = run(q, kv, sc, bt, L, 200, 3)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fmt,h_q,n,longest", [("bf16", 128, 30, 2000), ("bf16", 16, 5, 600), ("fp8", 16, 40, 5000), ("fp8", 64, 60, 3000)])
def test_an_output_on_sixteen_bytes(fmt, h_q, n, longest):
    """Outputs need 16-byte alignment, not more."""
    lens = [longest - 31 * b for b in range(n)]
    q, kv, sc, bt, L, want = problem(fmt, h_q, 1, lens, 1500, 3, seed=n)
    room = torch.empty(n * h_q * 512 + 8, dtype=torch.bfloat16, device="cuda")
    out = room[8:].view(n, 1, h_q, 512)
    assert out.data_ptr() % 32 == 16
    got = mla.window_decode(q, kv, bt, L, SCALE, window=1500, sinks=3, kv_scales=sc, out=out)
    assert mla.device_status() == 0
    check(*got, want, f"{fmt} at 16 bytes")


def test_calls_on_several_streams_at_once():
    """Every way a window is run, in turn on streams of their own with workspaces of their own."""
    cases = []
    for fmt, h_q, n, longest, window in (("bf16", 16, 4, 900, 300), ("fp8", 16, 100, 4000, 3500), ("bf16", 64, 40, 2000, 1500),
                                         ("bf16", 128, 20, 3000, 2500), ("fp8_token", 64, 30, 2500, 2000)):
        lens = [longest - 13 * b for b in range(n)]
        q, kv, sc, bt, L, want = problem(fmt, h_q, 1, lens, window, 9, seed=n)
        first = [t.clone() for t in run(q, kv, sc, bt, L, window, 9)]
        check(*first, want, f"{fmt} {h_q}x{n}")
        cases.append((q, kv, sc, bt, L, window, first, torch.cuda.Stream(),
                      torch.empty(mla.window_decode_workspace_size(n, h_q=h_q, s_q=1, is_fp8=fmt != "bf16"), dtype=torch.uint8,
                                  device="cuda")))
    torch.cuda.synchronize()
    results = [[] for _ in cases]
    for _ in range(10):
        for k, (q, kv, sc, bt, L, window, _, stream, ws) in enumerate(cases):
            results[k].append(mla.window_decode(q, kv, bt, L, SCALE, window=window, sinks=9, kv_scales=sc, workspace=ws,
                                                stream=stream))
    torch.cuda.synchronize()
    assert mla.device_status() == 0
    for case, got in zip(cases, results):
        for out, lse in got:
            assert torch.equal(out, case[6][0]) and torch.equal(lse, case[6][1])


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("h_q", [16, 40, 128])
@pytest.mark.parametrize("parts", [None, 30])
def test_lengths_below_zero_have_no_keys(fmt, h_q, parts):
    q, kv, sc, bt, L, want = problem(fmt, h_q, 2, (5, 130, 70, 300), 100, 4, seed=h_q)
    L[0], L[2] = -3, -2 ** 31
    with overrides(num_parts=parts):
        out, lse = run(q, kv, sc, bt, L, 100, 4)
    for b in (0, 2):
        assert (out[b] == 0).all() and (lse[b] == -float("inf")).all()
    keep = [1, 3]
    check(out[keep], lse[keep], tuple(w[keep] for w in want), f"{fmt} {h_q}")
