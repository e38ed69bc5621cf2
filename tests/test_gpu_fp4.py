"""The FP4 cache on the GPU: stores, reads and windowed decode against 64-bit references."""
import numpy as np
import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from fp4_reference import ROW, Fp4Cache, quantise, rows_of, stored
from gpu_helpers import Guarded, check_guards, guarded_tensor, overrides
from paged_reference import attend, check, i32, table
from test_gpu_window import problem, seen

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5
PAGE = 64


def edge_rows(g):
    """Latents and RoPE values where the format's rules meet: ties, block maxima at 6 * 2^k and beside it,
    zeros of both signs, blocks out of the scales' range, infinities."""
    x = torch.randn(40, 576, generator=g, device="cuda")
    x[0] = 0.0
    x[1, :512] = -0.0
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4, device="cuda")
    for k, e in enumerate(range(-13, 14, 2)):
        x[2 + k, :32] = ties * 2.0 ** e
        x[2 + k, 32:64] = -ties * 2.0 ** e
        x[2 + k, 64:96] = ties * 2.0 ** e * (1 + 2.0 ** -7)
        x[2 + k, 96:128] = ties * 2.0 ** e * (1 - 2.0 ** -8)
    x[20, :512] *= 1e-6
    x[21, :512] *= 1e-3
    x[22, :512] *= 1e6
    x[23, :512] *= 4e4
    x[24, 5] = float("inf")
    x[24, 70] = -float("inf")
    x[25, :512] = torch.exp2(torch.randint(-30, 30, (512,), generator=g, device="cuda").float())
    x[26, :512] = 2.0 ** -126
    x[27, :512] = 2.0 ** -133  # (a bf16 subnormal)
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("n,pad", [(1, 0), (40, 3), (127, 1), (5001, 50), (40000, 9)])
@pytest.mark.parametrize("width", [576, 2112])
def test_store(n, pad, width):
    g = torch.Generator("cuda").manual_seed(n)
    x = torch.randn(n, width, generator=g, device="cuda").to(torch.bfloat16)
    x[:, -576:] = torch.cat([edge_rows(g), x[40:, -576:]])[:n] if n >= 40 else x[:, -576:]
    x = x[:, -576:]
    pages = -(-n // PAGE) + 3
    slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:n]
    slots[n - pad:] = -1 - torch.arange(pad, device="cuda")
    gk, kv = guarded_tensor((pages, PAGE, 1, ROW), torch.uint8)
    kv.copy_(torch.randint(0, 256, kv.shape, generator=g, device="cuda", dtype=torch.uint8))
    want = kv.clone().view(-1, ROW)
    keep = slots >= 0
    want[slots[keep]] = rows_of(*quantise(x[keep, :512]), x[keep, 512:])
    mla.cache_store(x[:, :512], x[:, 512:], slots.int(), kv)
    assert mla.device_status() == 0
    check_guards({"kv": gk}, "store")
    assert torch.equal(kv.view(-1, ROW), want)


def test_store_nan_and_bad_slots():
    x = torch.ones(4, 576, device="cuda", dtype=torch.bfloat16)
    x[0, 3] = float("nan")
    kv = torch.zeros(2, PAGE, 1, ROW, dtype=torch.uint8, device="cuda")
    mla.cache_store(x[:, :512], x[:, 512:], i32([5, 128, 7, 2 ** 31 - 1]), kv)
    assert mla.device_status() == mla.DEVICE_BAD_PAGE
    back = mla.cache_load(kv, i32([[0]]), i32([0, 8]), 8)
    assert back[5, 3] == 6 * 0.25 and back[5, 4] == 1 and back[7, 0] == 1  # amax 1: scale 1/4
    assert mla.device_status() == 0
    assert (kv.view(-1, ROW)[128 - 64:] == 0).all()


FORMATS = ["bf16", "fp8", "fp8_token", "fp4"]


def cache_of(fmt, seed, pages):
    from paged_reference import Cache
    return Fp4Cache(fmt, seed, pages) if fmt == "fp4" else Cache(fmt, seed, pages)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,starts", [((1,), (0,)), ((5, 0, 0, 64, 1, 700, 0), (0, 5, 3, 63, 64, 65, 0)),
                                         ((0, 0, 3), (9, 9, 9)), ((2000, 1, 3000), None),
                                         (tuple(range(300)), tuple(range(300, 0, -1))), ((9000, 9000, 30), (1, 0, 70))])
@pytest.mark.parametrize("pad", [0, 7])
def test_load(fmt, lens, starts, pad):
    at = starts or (0,) * len(lens)
    cache = cache_of(fmt, 3, sum(-(-(a + n) // PAGE) for a, n in zip(at, lens)) + 2)
    want, ids = [], []
    for a, n in zip(at, lens):
        values, pages = cache.put(a + n)
        want.append(values[a:])
        ids.append(pages)
    kv, sc = cache.tensors() if fmt != "fp4" else (cache.raw.view(-1, PAGE, 1, ROW), None)
    total = sum(lens)
    g, out = guarded_tensor((total + pad, 576), torch.bfloat16)
    off = i32(np.concatenate([[0], np.cumsum(lens)]))
    got = mla.cache_load(kv, table(ids), off, total + pad, starts=i32(starts) if starts else None, kv_scales=sc, out=out)
    assert mla.device_status() == 0
    assert got.data_ptr() == out.data_ptr()
    check_guards({"out": g}, "load")
    assert torch.equal(got[:total].double(), torch.cat(want))
    assert (got[total:].view(torch.uint8) == 0xA5).all()  # rows behind the last request stay
    # offsets past the rows of out
    if total > 5:
        short = mla.cache_load(kv, table(ids), off, total - 5, starts=i32(starts) if starts else None, kv_scales=sc)
        assert torch.equal(short.double(), torch.cat(want)[:total - 5])
    assert mla.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_load_of_missing_pages(fmt):
    cache = cache_of(fmt, 5, 9)
    values, ids = cache.put(400)
    kv, sc = cache.tensors() if fmt != "fp4" else (cache.raw.view(-1, PAGE, 1, ROW), None)
    ids[2], ids[4] = -1, 9
    got = mla.cache_load(kv, table([ids]), i32([0, 500]), 500, kv_scales=sc)  # (and positions past the table)
    assert mla.device_status() == mla.DEVICE_BAD_PAGE
    want = torch.cat([values, torch.zeros(100, 576, device="cuda")])
    for pg in (2, 4):
        want[pg * PAGE:(pg + 1) * PAGE] = 0
    assert torch.equal(got[:400].double(), want[:400].double())
    assert (got[448:] == 0).all()  # (those between are slots of the last page that hold no token)
    got = mla.cache_load(kv, table([ids]), i32([0, 3]), 3, starts=i32([-2]), kv_scales=sc)
    assert mla.device_status() == mla.DEVICE_BAD_PAGE
    assert torch.equal(got.double(), torch.cat([torch.zeros(2, 576, device="cuda").double(), values[:1]]))


def test_bytes_that_no_store_writes_are_finite():
    # any byte is read as some finite latent value, the same by both readers
    g = torch.Generator("cuda").manual_seed(1)
    kv = torch.randint(0, 256, (3, PAGE, 1, ROW), generator=g, device="cuda", dtype=torch.uint8)
    kv[..., 272:] = torch.randn(3, PAGE, 1, 64, generator=g, device="cuda").to(torch.bfloat16).view(torch.uint8)
    rows = mla.cache_load(kv, i32([[0, 1, 2]]), i32([0, 192]), 192)
    assert torch.isfinite(rows).all()
    q = torch.zeros(1, 1, 16, 576, device="cuda", dtype=torch.bfloat16)  # the mean of the values
    out, lse = mla.window_decode(q, kv, i32([[0, 1, 2]]), i32([192]), SCALE, window=1 << 30)
    want = rows[:, :512].double().mean(0)
    mag = rows[:, :512].double().abs().mean(0)
    assert ((out[0, 0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * mag).all()
    assert (lse - np.log2(192)).abs().max() < 2.0 ** -18
    assert mla.device_status() == 0


# --------------------------------------------------------------------------- decode
def run(q, kv, sc, bt, lens, window, sinks, flags=0, **kw):
    b, s, h, _ = q.shape
    g_out, g_lse = Guarded(b * s * h * 1024), Guarded(b * s * h * 4)
    g_ws = Guarded(mla.window_decode_workspace_size(b, h_q=h, s_q=s, is_fp8=False, is_fp4=True))
    g_ws.body.fill_(0xFF)
    out, lse = mla.window_decode(q, kv.view(torch.uint8).view(-1, PAGE, 1, ROW), bt, lens, SCALE, window=window, sinks=sinks,
                                 out=g_out.view(torch.bfloat16, (b, s, h, 512)),
                                 lse=g_lse.view(torch.float32, (b, s, h)), workspace=g_ws.body, **kw)
    assert mla.device_status() == flags
    check_guards({"out": g_out, "lse": g_lse, "workspace": g_ws}, "window_decode over FP4 rows")
    return out, lse


def fp4_problem(h_q, s_q, lens, window, sinks, **kw):
    return problem("fp4", h_q, s_q, lens, window, sinks, make=Fp4Cache, **kw)


LENS = (0, 1, 5, 63, 64, 65, 127, 128, 129, 300, 641, 1000)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 0), (64, 64), (100, 10), (130, 65), (256, 129),
                                          (1000, 0), (200, 5000), (2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("h_q,s_q", [(16, 1), (128, 1), (24, 3)])
def test_window_and_sinks(h_q, s_q, window, sinks):
    q, kv, sc, bt, lens, want = fp4_problem(h_q, s_q, LENS, window, sinks, seed=window % 1000 + sinks % 1000)
    check(*run(q, kv, sc, bt, lens, window, sinks), want, f"{h_q}x{s_q} window {window} sinks {sinks}")


@pytest.mark.parametrize("h_q,s_q", [(1, 1), (8, 1), (8, 3), (20, 1), (32, 1), (33, 1), (64, 1), (16, 4), (65, 1), (40, 2),
                                     (128, 2), (96, 3), (100, 5), (1, 200), (512, 2)])
def test_row_counts(h_q, s_q):
    q, kv, sc, bt, lens, want = fp4_problem(h_q, s_q, (0, 2, 64, 190, 777), 150, 20, seed=h_q * 7 + s_q)
    check(*run(q, kv, sc, bt, lens, 150, 20), want, f"{h_q}x{s_q}")


@pytest.mark.parametrize("h_q", [16, 128])
@pytest.mark.parametrize("parts", [1, 2, 7, 40, 300])
def test_forced_splits(h_q, parts):
    q, kv, sc, bt, lens, want = fp4_problem(h_q, 2, (0, 700, 64, 1500, 3), 400, 70, seed=parts)
    with overrides(num_parts=parts):
        got = run(q, kv, sc, bt, lens, 400, 70)
    check(*got, want, f"{h_q} parts {parts}")


@pytest.mark.parametrize("h_q", [16, 128])
@pytest.mark.parametrize("n,longest", [(330, 900), (255, 200), (257, 200), (2500, 100), (14000, 40)])
def test_many_elements(h_q, n, longest):
    lens = [int(x) for x in np.random.default_rng(3).integers(0, longest, n)]
    if h_q == 128 and n > 3000:
        pytest.skip("covered at 16 heads")
    q, kv, sc, bt, L, want = fp4_problem(h_q, 1, lens, 200, 4, seed=5)
    check(*run(q, kv, sc, bt, L, 200, 4), want, f"{h_q}")


@pytest.mark.parametrize("h_q", [16, 128])
def test_an_unusable_page_is_flagged_and_masked(h_q):
    lens, window, sinks = (900, 500), 300, 64
    q, kv, sc, bt, L, _ = fp4_problem(h_q, 1, lens, window, sinks, seed=4)
    bt2 = bt.clone()
    bt2[0, 900 // 64 - 1] = kv.numel()
    got = run(q, kv, sc, bt2, L, window, sinks, flags=mla.DEVICE_BAD_PAGE)
    whole = run(q, kv, sc, bt, L, window, sinks)
    assert torch.isfinite(got[0]).all()
    assert torch.allclose(got[1][1], whole[1][1], rtol=0, atol=2.0 ** -18)
    assert (got[1][0] < whole[1][0]).all()
    run(q, kv, sc, bt[:, :14].contiguous(), L, window, 0, flags=mla.DEVICE_BAD_PAGE)  # a table too short


@pytest.mark.parametrize("h_q,s_q,window", [(16, 1, 1 << 30), (128, 1, 1 << 30), (128, 2, 1000), (40, 1, 700)])
def test_repeated_calls_are_equal(h_q, s_q, window):
    # pages that lie in L2 come back faster than they are read: no word of a page may be the next one's
    lens = [int(x) for x in np.random.default_rng(7).integers(50, 5000, 40)]
    q, kv, sc, bt, L, want = fp4_problem(h_q, s_q, lens, window, 16, seed=11)
    first = run(q, kv, sc, bt, L, window, 16)
    check(*first, want, f"{h_q}x{s_q}")
    for _ in range(200):
        out, lse = mla.window_decode(q, kv.view(torch.uint8).view(-1, PAGE, 1, ROW), bt, L, SCALE, window=window, sinks=16)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert mla.device_status() == 0


def test_captured_calls_and_other_streams():
    q, kv, sc, bt, L, want = fp4_problem(32, 1, (700, 64, 3000), 500, 4, seed=12)
    kv = kv.view(torch.uint8).view(-1, PAGE, 1, ROW)
    first = run(q, kv, sc, bt, L, 500, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = mla.window_decode(q, kv, bt, L, SCALE, window=500, sinks=4)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [mla.window_decode(q, kv, bt, L, SCALE, window=500, sinks=4, stream=s) for s in streams for _ in range(5)]
    graph.replay()
    torch.cuda.synchronize()
    for o, z in [*got, (out, lse)]:
        assert torch.equal(o, first[0]) and torch.equal(z, first[1])


def test_refusals_name_the_argument():
    q, kv, sc, bt, L, _ = fp4_problem(16, 1, (100,), 50, 0, seed=1)
    kv = kv.view(torch.uint8).view(-1, PAGE, 1, ROW)
    with pytest.raises(ValueError, match="kv_scales given with an FP4 kvcache"):
        mla.window_decode(q, kv, bt, L, SCALE, window=5, kv_scales=torch.ones(kv.shape[:2], device="cuda"))
    with pytest.raises(ValueError, match="does not take an FP4 kvcache"):
        mla.shared_prefix_decode(q, kv, bt[0], L, bt, L, SCALE)
    with pytest.raises(ValueError, match="page_size"):
        mla.window_decode(q, kv.view(-1, 32, 1, ROW), bt, L, SCALE, window=5)
    with pytest.raises(ValueError, match="out must be"):
        mla.cache_load(kv, bt, i32([0, 5]), 5, out=torch.empty(4, 576, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="row_offsets must have"):
        mla.cache_load(kv, bt, i32([0, 5, 6]), 5)
    with pytest.raises(ValueError, match="starts must have"):
        mla.cache_load(kv, bt, i32([0, 5]), 5, starts=i32([0, 1]))


@pytest.mark.parametrize("h_q", [16, 128])
def test_watchdog_reports_an_expired_wait(h_q):
    from gpu_helpers import env
    q, kv, sc, bt, L, want = fp4_problem(h_q, 1, (900, 300), 1 << 30, 0, seed=2)
    for parts in (None, 3):  # clusters, a schedule
        with env(MLA_WATCHDOG_NS=20_000_000), overrides(debug_stall=True, num_parts=parts):
            mla.window_decode(q, kv.view(torch.uint8).view(-1, PAGE, 1, ROW), bt, L, SCALE, window=1 << 30)
            torch.cuda.synchronize()
        assert mla.device_status() & mla.DEVICE_TIMEOUT
        check(*run(q, kv, sc, bt, L, 1 << 30, 0), want, "after a timeout")


def test_rows_that_are_not_finite_stay_alone():
    q, kv, sc, bt, L, _ = fp4_problem(16, 1, (300, 700), 1 << 30, 0, seed=3)
    want = run(q, kv, sc, bt, L, 1 << 30, 0)
    q[0, 0, 5, 100] = float("nan")
    q[1, 0, 7, 570] = float("inf")
    out, lse = run(q, kv, sc, bt, L, 1 << 30, 0)
    keep = torch.ones(2, 1, 16, dtype=torch.bool, device="cuda")
    keep[0, 0, 5] = keep[1, 0, 7] = False
    assert torch.isnan(out[~keep]).all() and torch.isnan(lse[~keep]).all()
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


@pytest.mark.parametrize("spread", [1e-3, 20.0])
def test_query_magnitudes(spread):
    # rows of q of any size, values of a row 2^12 apart: split into two 8-bit terms
    q, kv, sc, bt, L, _ = fp4_problem(16, 1, (500,), 1 << 30, 0, seed=4)
    q.mul_(spread * torch.exp2(torch.randint(-12, 1, q.shape, device="cuda").float()).to(torch.bfloat16))
    out, lse = run(q, kv, sc, bt, L, 1 << 30, 0)
    rows = mla.cache_load(kv.view(torch.uint8).view(-1, PAGE, 1, ROW), bt, i32([0, 500]), 500).double()
    want_out, want_lse, mean = attend(q[0, 0], rows, SCALE)
    # a term of q is off by 2^-18 of its row's largest value, 576 of them meet keys of about one, then the scale
    off = 2.0 ** -18 * q.abs().max().item() * 576 * rows.abs().mean().item() * SCALE
    assert (lse[0, 0].double() - want_lse).abs().max().item() <= off + 2.0 ** -9
    # A weight is held in three E5M2 terms at 2^8 or more times its share of the row's largest one; E5M2's
    # smallest number is 2^-16, half of it 2^-17, so a weight is off by no more than the larger of 2^-9 of
    # itself and 2^-17 / 2^8 = 2^-25 of the largest.  Where q is this large nearly all of a row's weight
    # is one key's, and a dim that is 0 there is made of the small ones alone.
    least = 2.0 ** -25 * rows[:, :512].abs().sum(0)
    assert ((out[0, 0].double() - want_out).abs()
            <= (2.0 ** -8 + 2 * off + 2.0 ** -9) * mean + 2.0 ** -8 * want_out.abs() + least).all()


def test_weights_far_below_the_largest():
    # one key 2^14 above 6000 others, which together have a third of its weight
    n = 6000
    cache = Fp4Cache("fp4", 5, -(-n // PAGE) + 1)
    values, ids = cache.put(n)
    kv = cache.raw.view(-1, PAGE, 1, ROW)
    q = torch.zeros(1, 1, 16, 576, device="cuda", dtype=torch.bfloat16)
    top = values[1234, 512:]
    q[0, 0, :, 512:] = top.to(torch.bfloat16)
    scale = (14.2 * np.log(2.0)) / float(top @ top)
    rows = torch.cat([values[:, :512], torch.zeros(n, 64, device="cuda", dtype=torch.float64)], 1)
    raw = cache.raw.view(-1, ROW)
    slots = torch.tensor(ids, device="cuda").repeat_interleave(PAGE)[:n] * PAGE + torch.arange(n, device="cuda") % PAGE
    raw[slots, 272:] = 0  # the others' RoPE values: scores of 0
    raw[slots[1234], 272:] = top.to(torch.bfloat16).view(torch.uint8)
    rows[1234, 512:] = top.to(torch.bfloat16).double()
    out, lse = mla.window_decode(q, kv, table([ids]), i32([n]), scale, window=1 << 30)
    want = attend(q[0, 0], rows, scale)
    assert abs(float(torch.exp2(want[1][0] - 14.2)) - 1.32) < 0.02
    check(out, lse, tuple(w[None, None] for w in want), "small weights")
    assert mla.device_status() == 0
