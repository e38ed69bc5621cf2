"""Page assignment and cache store through slots on the GPU, against definitions written out with
Python integers and 64-bit floats."""
import numpy as np
import pytest
import torch

import paged_mla_decode_07_gb300 as mla

from gpu_helpers import Guarded, check_guards

pytestmark = pytest.mark.gpu

PAGE = 64


def ref_assign(old, new, free, cursor, table, num_tokens, num_pages):
    """(table, seqlens, offsets, slots, next_cursor, no_room, bad_page) by walking the requests."""
    table = table.copy()
    stride = table.shape[1]
    at = min(max(cursor, 0), len(free))
    slots, offsets, lens, no_room, bad = [], [0], [], False, False
    for b in range(len(old)):
        o, n = max(int(old[b]), 0), max(int(new[b]), 0)
        pages = {}
        for pg in range(-(-o // PAGE), -(-(o + n) // PAGE)):
            if pg >= stride:
                no_room = True
                pages[pg] = -1
                continue
            if at < len(free):
                pages[pg] = int(free[at])
            else:
                no_room, pages[pg] = True, -1
            at += 1
            if pages[pg] >= num_pages or (pages[pg] < 0 and at <= len(free)):
                bad, pages[pg] = True, -1
            table[b, pg] = pages[pg]
        for pos in range(o, o + n):
            pg = pos // PAGE
            page = pages.get(pg, int(table[b, pg]) if pg < stride else -1)
            if pg not in pages and (page < 0 or page >= num_pages):
                if pg < stride:
                    bad = True
                page = -1
            slots.append(page * PAGE + pos % PAGE if page >= 0 else -1)
        offsets.append(offsets[-1] + n)
        lens.append(o + n)
    no_room = no_room or len(slots) > num_tokens
    slots = (slots + [-1] * num_tokens)[:num_tokens]
    return table, lens, offsets, slots, min(at, len(free)), no_room, bad


def i32(x):
    return torch.tensor(np.asarray(x, np.int64), dtype=torch.int32, device="cuda")


def guarded_i32(values):
    values = np.ascontiguousarray(values, np.int32)
    g = Guarded(max(4, values.nbytes))
    t = g.view(torch.int32, (-1,))[:values.size].view(values.shape)
    t.copy_(torch.from_numpy(values))
    return g, t


def run_assign(old, new, free, cursor, table, num_tokens, num_pages, in_place=False):
    batch = len(old)
    g = {}
    g["table"], t_table = guarded_i32(table)
    g["lens"], t_lens = guarded_i32(old if in_place else np.full(batch, -7))
    g["offsets"], t_off = guarded_i32(np.full(batch + 1, -7))
    g["slots"], t_slots = guarded_i32(np.full(num_tokens, -7))
    g["cursor"], t_cur = guarded_i32([cursor if in_place else -7])
    got = mla.assign_pages(t_lens if in_place else i32(old), i32(new), i32(free), t_cur if in_place else i32([cursor]),
                           t_table, num_tokens, num_pages=num_pages, cache_seqlens=t_lens, row_offsets=t_off,
                           slot_map=t_slots, next_cursor=t_cur)
    flags = mla.device_status()
    check_guards(g, "assign_pages")
    assert [x.data_ptr() for x in got] == [t_lens.data_ptr(), t_off.data_ptr(), t_slots.data_ptr(), t_cur.data_ptr()]
    return t_table.cpu().numpy(), t_lens.tolist(), t_off.tolist(), t_slots.tolist(), int(t_cur[0]), flags


def check_assign(old, new, free, cursor, table, num_tokens, num_pages, in_place=False):
    want = ref_assign(old, new, free, cursor, table, num_tokens, num_pages)
    got = run_assign(old, new, free, cursor, table, num_tokens, num_pages, in_place)
    assert np.array_equal(got[0], want[0])
    assert got[1] == want[1] and got[2] == want[2] and got[3] == want[3] and got[4] == want[4]
    assert got[5] == (mla.DEVICE_NO_ROOM if want[5] else 0) | (mla.DEVICE_BAD_PAGE if want[6] else 0)


def problem(rng, batch, old_hi, new_lo, new_hi, spare_cols=2, spare_free=5, start=3):
    old = rng.integers(0, old_hi + 1, batch)
    new = rng.integers(new_lo, new_hi + 1, batch)
    have, want = -(-old // PAGE), -(-(old + new) // PAGE)
    pool = rng.permutation(int(want.sum()) + spare_free)
    table = np.full((batch, int(want.max()) + spare_cols), -1)
    at = 0
    for b in range(batch):
        table[b, :have[b]] = pool[at:at + have[b]]
        at += have[b]
    free = np.concatenate([rng.integers(0, len(pool), start), pool[at:]])
    return old, new, free, start, table, len(pool)


@pytest.mark.parametrize("batch,old_hi,new_lo,new_hi,pad", [
    (1, 0, 1, 1, 0), (1, 63, 1, 1, 0), (1, 64, 1, 1, 3), (3, 500, 0, 0, 5), (3, 500, 0, 0, 0), (64, 4000, 1, 1, 0),
    (64, 4000, 0, 2, 1), (5, 200, 0, 700, 2), (33, 1000, 60, 70, 0), (700, 300, 0, 5, 7), (2000, 128, 1, 1, 0),
    (40, 2000, 0, 1500, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_assign_pages(batch, old_hi, new_lo, new_hi, pad, in_place):
    rng = np.random.default_rng(batch * 1000 + old_hi + new_hi)
    old, new, free, start, table, pool = problem(rng, batch, old_hi, new_lo, new_hi)
    check_assign(old, new, free, start, table, int(new.sum()) + pad, pool, in_place)


@pytest.mark.parametrize("old", [0, 1, 63, 64, 65, 127, 128])
@pytest.mark.parametrize("new", [0, 1, 2, 63, 64, 65, 129])
def test_assign_pages_at_page_edges(old, new):
    rng = np.random.default_rng(old * 200 + new)
    check_assign([old, 5, old], [new, 1, new], rng.permutation(40), 0, np.full((3, 6), 39) + np.arange(3)[:, None] * 0,
                 2 * new + 1, 40)


def test_assign_pages_at_the_largest_batch():
    rng = np.random.default_rng(5)
    old, new, free, start, table, pool = problem(rng, 16384, 200, 0, 3)
    check_assign(old, new, free, start, table, int(new.sum()) + 11, pool)
    check_assign(old, new, free, start, table, int(new.sum()) + 11, pool, in_place=True)


def test_assign_pages_reports_what_does_not_fit():
    rng = np.random.default_rng(9)
    old, new, free, start, table, pool = problem(rng, 12, 300, 0, 300)
    tokens = int(new.sum())
    check_assign(old, new, free[: start + 4], start, table, tokens, pool)          # the free list ends
    check_assign(old, new, free[:0], 0, table, tokens, pool)                       # there is none
    check_assign(old, new, free, start, table[:, :4], tokens, pool)                # the table rows end
    check_assign(old, new, free, start, table, tokens - 5, pool)                   # the slot map ends
    check_assign(old, new, free, start, table, tokens, pool - 9)                   # pages outside the cache
    check_assign(-old, new, free, -4, table, tokens, pool)                         # negative lengths, cursor
    check_assign(old, -new, free, 10 ** 6, table, 10, pool)                        # nothing new, cursor past the end


def test_assign_pages_in_a_replayed_graph_advances_in_place():
    rng = np.random.default_rng(4)
    old, new, free, start, table, pool = problem(rng, 9, 200, 1, 1, spare_cols=6, spare_free=60)
    lens, cur, tab = i32(old), i32([start]), i32(table)
    new_t, free_t = i32(new), i32(free)
    off = torch.empty(10, dtype=torch.int32, device="cuda")
    slots = torch.empty(12, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mla.assign_pages(lens, new_t, free_t, cur, tab, 12, num_pages=pool, cache_seqlens=lens, row_offsets=off,
                         slot_map=slots, next_cursor=cur)
    torch.cuda.synchronize()
    old = np.array(old)
    for _ in range(200):
        graph.replay()
        torch.cuda.synchronize()
        table, want_lens, _, want_slots, start, no_room, _ = ref_assign(old, new, free, start, table, 12, pool)
        assert lens.tolist() == want_lens and slots.tolist() == want_slots and int(cur[0]) == start
        assert np.array_equal(tab.cpu().numpy(), table)
        assert mla.device_status() == (mla.DEVICE_NO_ROOM if no_room else 0)
        old = np.array(want_lens)


# ------------------------------------------------------------------ cache store
ROW = {"fp8": 656, "fp8_token": 640}


def e4m3_nearest(v):
    """Nearest E4M3 magnitude code (ties to even, saturating) of non-negative float64 values."""
    grid = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    hi = np.clip(np.searchsorted(grid, v), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dl, dh = v - grid[lo], grid[hi] - v
    pick_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (v >= grid[126])
    return np.where(pick_hi, np.where(v >= grid[126], 126, hi), lo).astype(np.uint8)


def ref_rows(latent, rope, fmt):
    """Row bytes [n, row] and scales [n] of float32-exact inputs."""
    n = latent.shape[0]
    rope_bytes = rope.contiguous().view(torch.uint8).numpy().reshape(n, 128)
    if fmt == "bf16":
        lat = latent.contiguous().view(torch.uint8).numpy().reshape(n, 1024)
        return np.concatenate([lat, rope_bytes], 1), None
    x = latent.float().numpy().reshape(n, 4 if fmt == "fp8" else 1, -1)
    amax = np.abs(x).max(-1, keepdims=True)
    scale = np.where(amax > 0, amax / np.float32(448), np.float32(1)).astype(np.float32)
    quot = (x / scale).astype(np.float32)  # float32 division, as the format defines
    codes = e4m3_nearest(np.abs(quot).astype(np.float64)) | (np.signbit(quot).astype(np.uint8) << 7)
    codes = codes.reshape(n, 512)
    s = scale.reshape(n, -1)
    if fmt == "fp8":
        return np.concatenate([codes, s.view(np.uint8).reshape(n, 16), rope_bytes], 1), None
    return np.concatenate([codes, rope_bytes], 1), s[:, 0]


def store_case(rng, n, pages, fmt, width):
    g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    x = torch.randn(n, max(width, 576), generator=g) * torch.exp2(torch.randint(-20, 12, (n, 1), generator=g).float())
    if n > 2:
        x[1] = 0
        x[2, 200:] *= 2.0 ** -60
    x = x.to(torch.bfloat16).cuda()
    if width:
        latent, rope = x[:, width - 576:width - 64], x[:, width - 64:]
    else:
        latent, rope = x[:, :512].contiguous(), x[:, 512:].contiguous()
    slots = rng.permutation(pages * PAGE)[:n]
    return latent, rope, slots


def run_store(latent, rope, slots, pages, fmt, flags=0):
    row = 1152 if fmt == "bf16" else ROW[fmt]
    kv_g, sc_g = Guarded(pages * PAGE * row), Guarded(pages * PAGE * 4)
    kv_g.body.fill_(0x5B)
    sc_g.body.fill_(0x5B)
    kv = kv_g.view(torch.bfloat16, (pages, PAGE, 1, 576)) if fmt == "bf16" else kv_g.view(torch.uint8, (pages, PAGE, 1, row))
    sc = sc_g.view(torch.float32, (pages, PAGE))
    mla.cache_store(latent, rope, i32(slots), kv, kv_scales=sc if fmt == "fp8_token" else None)
    assert mla.device_status() == flags
    check_guards({"kv": kv_g, "scales": sc_g}, "cache_store")
    want = np.full((pages * PAGE, row), 0x5B, np.uint8)
    want_s = np.full(pages * PAGE * 4, 0x5B, np.uint8).view(np.float32)
    rows, scales = ref_rows(latent.cpu(), rope.cpu(), fmt)
    ok = (np.asarray(slots) >= 0) & (np.asarray(slots) < pages * PAGE)
    want[np.asarray(slots)[ok]] = rows[ok]
    if scales is not None:
        want_s[np.asarray(slots)[ok]] = scales[ok]
    assert np.array_equal(kv_g.body.cpu().numpy().reshape(-1, row), want)
    assert np.array_equal(sc_g.body.cpu().numpy(), want_s.view(np.uint8))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("n,width", [(1, 0), (2, 576), (7, 0), (64, 2112), (1000, 0), (9001, 584), (40000, 0)])
def test_cache_store_matches_the_format(fmt, n, width):
    rng = np.random.default_rng(n)
    pages = -(-n // PAGE) + 3
    latent, rope, slots = store_case(rng, n, pages, fmt, width)
    run_store(latent, rope, slots, pages, fmt)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_token"])
def test_cache_store_skips_padding_and_flags_slots_past_the_cache(fmt):
    rng = np.random.default_rng(3)
    latent, rope, slots = store_case(rng, 50, 2, fmt, 0)
    slots[10:20] = -1
    slots[30] = -12345
    run_store(latent, rope, slots, 2, fmt)
    slots[40], slots[41] = 2 * PAGE, 2 ** 31 - 1
    run_store(latent, rope, slots, 2, fmt, flags=mla.DEVICE_BAD_PAGE)


@pytest.mark.parametrize("fmt", ["fp8", "fp8_token"])
@pytest.mark.parametrize("power", [-133, -126, -110, -98, -97, -90, -82, -81, -60, 60, 110, 126])
def test_cache_store_at_the_ends_of_the_range(fmt, power):
    # scales around the limits between which the quotients are refined from a reciprocal
    rng = np.random.default_rng(power + 200)
    latent, rope, slots = store_case(rng, 40, 2, fmt, 0)
    g = torch.Generator().manual_seed(power + 300)
    m = torch.rand(40, 512, generator=g).double() * torch.where(torch.rand(40, 512, generator=g) < 0.5, -1.0, 1.0)
    m[:, ::3] *= 2.0 ** -7
    m[:, ::5] *= 2.0 ** -14
    latent.copy_((m * 2.0 ** power).to(torch.bfloat16))
    run_store(latent, rope, slots, 2, fmt)


def test_cache_store_of_no_tokens_is_a_no_op():
    latent, rope, _ = store_case(np.random.default_rng(1), 1, 1, "bf16", 0)
    run_store(latent[:0], rope[:0], np.zeros(0, int), 2, "bf16")


def test_cache_store_special_values_stay_in_their_token():
    # a NaN or an infinity spoils its own scale tile, no other token and no RoPE value
    latent, rope, slots = store_case(np.random.default_rng(8), 12, 1, "fp8", 0)
    latent[4, 3], latent[6, 300] = float("nan"), float("inf")
    kv = torch.zeros(1, PAGE, 1, 656, dtype=torch.uint8, device="cuda")
    mla.cache_store(latent, rope, i32(slots), kv)
    assert mla.device_status() == 0
    rows, _ = ref_rows(torch.nan_to_num(latent.cpu(), posinf=1.0), rope.cpu(), "fp8")
    got = kv.view(PAGE, 656).cpu().numpy()[slots]
    keep = [i for i in range(12) if i not in (4, 6)]
    assert np.array_equal(got[keep], rows[keep])
    assert np.array_equal(got[[4, 6], 528:], rows[[4, 6], 528:])  # RoPE parts
    assert np.array_equal(got[4, 128:512], rows[4, 128:512]) and np.array_equal(got[6, :256], rows[6, :256])
    assert got[4, 3] & 0x7F == 0x7F  # the NaN is stored as one


def test_cache_store_equals_the_table_driven_store():
    # the same tokens through mla_fp8_cache_store's block table and through the slots of assign_pages
    rng = np.random.default_rng(21)
    old, new, free, start, table, pool = problem(rng, 7, 300, 0, 90)
    n = int(new.sum())
    x = torch.randn(n, 576, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(torch.bfloat16)
    tab = i32(table)
    lens, off, slots, _ = mla.assign_pages(i32(old), i32(new), i32(free), i32([start]), tab, n, num_pages=pool)
    a = torch.zeros(pool, PAGE, 1, 656, dtype=torch.uint8, device="cuda")
    b = torch.zeros_like(a)
    mla.cache_store(x[:, :512], x[:, 512:], slots, a)
    mla.fp8_cache_store(x, off, i32(old), tab, b)
    assert mla.device_status() == 0
    assert torch.equal(a, b)


def test_store_on_a_side_stream():
    rng = np.random.default_rng(2)
    latent, rope, slots = store_case(rng, 300, 6, "fp8", 0)
    want = torch.zeros(6, PAGE, 1, 656, dtype=torch.uint8, device="cuda")
    mla.cache_store(latent, rope, i32(slots), want)
    got, s = torch.zeros_like(want), i32(slots)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    mla.cache_store(latent, rope, s, got, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    got.zero_()
    torch.cuda.synchronize()
    mla.cache_store(latent, rope, s, got, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want)
    assert mla.device_status() == 0
