"""Shared-prefix decode on the GPU against a 64-bit reference."""
import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from gpu_helpers import Guarded, check_guards, overrides
from paged_reference import Cache, attend, check, i32, table

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5


@pytest.fixture(params=["any", "blocks"], autouse=True)
def path(request):
    """Every test as the call chooses its kernels, and with the blocks of 128 rows that large calls take."""
    if request.param == "any":
        yield
    else:
        with overrides(num_parts=60):
            yield


def problem(fmt, h_q, s_q, prefix, own, causal, seed=0):
    cache = Cache(fmt, seed, -(-prefix // 64) + sum(-(-L // 64) for L in own) + 3)
    g = torch.Generator("cuda").manual_seed(seed + 1)
    q = torch.randn(len(own), s_q, h_q, 576, generator=g, device="cuda").to(torch.bfloat16)
    shared, prefix_ids = cache.put(prefix)
    rows, want = [], []
    for b, L in enumerate(own):
        values, ids = cache.put(L)
        rows.append(ids)
        for i in range(s_q):
            n = max(0, min(L, L - s_q + i + 1)) if causal else L
            want.append(attend(q[b, i], torch.cat([shared, values[:n]]), SCALE))
    want = tuple(torch.stack([w[k] for w in want]).view(len(own), s_q, h_q, *([512] if k != 1 else [])) for k in range(3))
    kv, sc = cache.tensors()
    return q, kv, sc, table([prefix_ids], width=max(1, len(prefix_ids)))[0], i32([prefix]), table(rows), i32(own), want


def run(q, kv, sc, pt, plen, bt, lens, causal, flags=0, **kw):
    b, s, h, _ = q.shape
    g_out, g_lse = Guarded(b * s * h * 1024), Guarded(b * s * h * 4)
    g_ws = Guarded(mla.shared_prefix_decode_workspace_size(b, h_q=h, s_q=s, prefix_table_len=pt.shape[0],
                                                           is_fp8=kv.dtype == torch.uint8))
    g_ws.body.fill_(0xFF)
    out, lse = mla.shared_prefix_decode(q, kv, pt, plen, bt, lens, SCALE, is_causal=causal, kv_scales=sc,
                                        out=g_out.view(torch.bfloat16, (b, s, h, 512)),
                                        lse=g_lse.view(torch.float32, (b, s, h)), workspace=g_ws.body, **kw)
    assert mla.device_status() == flags
    check_guards({"out": g_out, "lse": g_lse, "workspace": g_ws}, "shared_prefix_decode")
    return out, lse


OWN = (0, 1, 63, 64, 65, 130, 300)


@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 128, 129, 200, 1000, 2500])
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("h_q,s_q,causal", [(16, 1, False), (128, 1, True), (20, 2, True), (24, 2, False)])
def test_prefix_lengths(fmt, h_q, s_q, causal, prefix):
    case = problem(fmt, h_q, s_q, prefix, OWN, causal, seed=prefix + h_q)
    check(*run(*case[:7], causal), case[7], f"{fmt} {h_q}x{s_q} prefix {prefix}")


@pytest.mark.parametrize("h_q,s_q", [(1, 1), (8, 3), (32, 1), (33, 1), (64, 2), (65, 1), (128, 2), (96, 3), (1, 200), (512, 2)])
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_row_counts(fmt, h_q, s_q):
    case = problem(fmt, h_q, s_q, 333, (5, 0, 100), True, seed=h_q * 5 + s_q)
    check(*run(*case[:7], True), case[7], f"{fmt} {h_q}x{s_q}")


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("parts", [1, 2, 9, 60, 300])
def test_forced_splits(fmt, parts):
    case = problem(fmt, 40, 2, 1500, (0, 700, 64, 200, 3), True, seed=parts)
    with overrides(num_parts=parts):
        got = run(*case[:7], True)
    check(*got, case[7], f"{fmt} parts {parts}")


@pytest.mark.parametrize("fmt,h_q", [("bf16", 16), ("bf16", 128), ("fp8", 16), ("fp8_token", 64)])
@pytest.mark.parametrize("n,prefix", [(150, 1111), (1200, 100)])
def test_many_elements(fmt, h_q, n, prefix):
    # several problems per thread of the schedule that every CTA makes
    own = [(i * 37) % 190 for i in range(n)]
    case = problem(fmt, h_q, 1, prefix, own, True, seed=8)
    check(*run(*case[:7], True), case[7], f"{fmt} {h_q}")


def test_one_element_without_a_prefix_or_keys():
    case = problem("bf16", 16, 1, 0, (0,), True, seed=2)
    out, lse = run(*case[:7], True)
    assert (out == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_equals_dense_decode_over_the_joined_tables(fmt):
    # a prefix of whole pages: each element's table row is the prefix's pages and its own
    own = (5, 200, 64)
    q, kv, sc, pt, plen, bt, lens, want = problem(fmt, 16, 1, 640, own, False, seed=11)
    got = run(q, kv, sc, pt, plen, bt, lens, False)
    full = torch.cat([pt.expand(3, -1), bt], 1).contiguous()
    total = (lens + plen).int()
    sched, ns = mla.get_metadata(total, h_q=16, s_q=1, topk=0, is_fp8=fmt != "bf16")
    ref = mla.decode(q, kv, full, total, SCALE, sched, ns)
    assert mla.device_status() == 0
    # two evaluations of the same formula, each within check()'s bound of it
    assert (got[0].double() - ref[0].double()).abs().le(2 * ((2.0 ** -8 + 2.0 ** -9) * want[2] + 2.0 ** -8 * want[0].abs())).all()
    assert (got[1] - ref[1]).abs().max() <= 2.0 ** -8


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_unusable_pages_are_flagged_and_masked(fmt):
    case = problem(fmt, 16, 1, 300, (100, 20), False, seed=3)
    q, kv, sc, pt, plen, bt, lens, _ = case
    whole = run(*case[:7], False)
    pt2, bt2 = pt.clone(), bt.clone()
    pt2[1] = -5
    got = run(q, kv, sc, pt2, plen, bt, lens, False, flags=mla.DEVICE_BAD_PAGE)
    assert torch.isfinite(got[0]).all() and (got[1] < whole[1]).all()
    bt2[0, 0] = kv.shape[0]
    got = run(q, kv, sc, pt, plen, bt2, lens, False, flags=mla.DEVICE_BAD_PAGE)
    assert torch.isfinite(got[0]).all() and (got[1][0] < whole[1][0]).all()
    assert torch.allclose(got[1][1], whole[1][1], rtol=0, atol=2.0 ** -18)
    # a length past the prefix table: the missing pages are masked
    plen2 = plen + 64
    got = run(q, kv, sc, pt[:4].contiguous(), plen2, bt, lens, False, flags=0 if fmt == "none" else mla.DEVICE_BAD_PAGE)
    assert torch.isfinite(got[0]).all()


def test_repeated_runs_and_graph_replays_agree():
    case = problem("fp8", 64, 2, 700, (90, 13, 64), True, seed=6)
    q, kv, sc, pt, plen, bt, lens, _ = case
    first = [t.clone() for t in run(*case[:7], True)]
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    ws = torch.empty(mla.shared_prefix_decode_workspace_size(3, h_q=64, s_q=2, prefix_table_len=pt.shape[0], is_fp8=True),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.shared_prefix_decode(q, kv, pt, plen, bt, lens, SCALE, is_causal=True, out=out, lse=lse, workspace=ws)
    for _ in range(10):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    plen.fill_(65)
    lens.fill_(3)
    graph.replay()
    again = run(*case[:7], True)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("h_q", [16, 40, 128])
@pytest.mark.parametrize("more", [1, 64, 2 ** 31 - 1])
def test_lengths_past_the_tables(fmt, h_q, more):
    q, kv, sc, pt, plen, bt, lens, want = problem(fmt, h_q, 1, 192, (128, 128, 128), False, seed=h_q)
    far = i32([min(2 ** 31 - 1, 128 + more)] * 3)
    check(*run(q, kv, sc, pt, plen, bt, far, False, flags=mla.DEVICE_BAD_PAGE), want, f"{fmt} own")
    plen.fill_(min(2 ** 31 - 1, 192 + more))
    check(*run(q, kv, sc, pt, plen, bt, lens, True, flags=mla.DEVICE_BAD_PAGE), want, f"{fmt} prefix")


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("h_q,s_q", [(1, 1), (16, 1), (20, 2), (128, 1)])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_keys_that_are_not_finite_stay_in_their_element(fmt, h_q, s_q, bad):
    """Rows of several elements share a block of the products: one element's broken keys reach no other one."""
    own = (70, 130, 64, 5, 200, 1)
    q, kv, sc, pt, plen, bt, lens, want = problem(fmt, h_q, s_q, 300, own, False, seed=h_q)
    hit = 1
    for t in (3, 129):
        page, slot = int(bt[hit, t // 64]), t % 64
        if fmt == "bf16":
            kv.view(torch.int16)[page, slot, 0, 7 * t % 512] = 0x7FC0 if bad == "nan" else 0x7F80
        else:
            kv[page, slot, 0, 512:516].view(torch.float32).fill_(float(bad))
    out, lse = run(q, kv, sc, pt, plen, bt, lens, False)
    keep = [b for b in range(len(own)) if b != hit]
    check(out[keep], lse[keep], tuple(w[keep] for w in want), f"{fmt} {h_q} beside {bad}")
    assert bool(torch.isnan(out[hit]).any()) and not bool(torch.isfinite(lse[hit]).any() and bad == "nan")


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("h_q", [16, 40, 128])
def test_lengths_below_zero_have_no_keys(fmt, h_q):
    q, kv, sc, pt, plen, bt, lens, want = problem(fmt, h_q, 1, 100, (60, 130, 70), False, seed=h_q)
    lens[0], lens[2] = -1, -2 ** 31
    out, lse = run(q, kv, sc, pt, plen, bt, lens, False)
    check(out[1:2], lse[1:2], tuple(w[1:2] for w in want), f"{fmt} {h_q}")
    zero = lens.clone().fill_(0)
    empty = run(q, kv, sc, pt, plen, bt, zero, False)
    for b in (0, 2):  # (the pieces may be cut elsewhere)
        assert torch.allclose(lse[b], empty[1][b], rtol=0, atol=2.0 ** -18)
        assert torch.allclose(out[b].float(), empty[0][b].float(), rtol=2.0 ** -7, atol=2.0 ** -7)
    plen.fill_(-7)
    out, lse = run(q, kv, sc, pt, plen, bt, lens, False)
    assert (out[0] == 0).all() and (lse[2] == -float("inf")).all() and torch.isfinite(lse[1]).all()
