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
