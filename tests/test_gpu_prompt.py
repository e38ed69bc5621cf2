"""Attention over packed prompts on the GPU against a 64-bit reference."""
import math

import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from gpu_helpers import Guarded, check_guards, overrides
from paged_reference import check, i32

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


def inputs(h_q, h_kv, lens, seed=0, pad=0, gap=0, spread=1.0):
    """Packed q and keys of sequences of (queries, keys); `pad` rows behind the last sequence, `gap` more values
    between the rows of every tensor.  Keys and values that belong to no sequence are NaN."""
    g = torch.Generator("cuda").manual_seed(seed)
    nq, nk = sum(n for n, _ in lens), sum(m for _, m in lens)

    def rand(*shape):
        return (torch.randn(*shape, generator=g, device="cuda") * spread).to(torch.bfloat16)

    q = rand(nq + pad, h_q, 192 + gap)[..., :192]
    up = rand(nk + pad, h_kv, 256 + gap)
    rows = rand(nk + pad, 576 + gap)
    up[nk:], rows[nk:] = float("nan"), float("nan")
    k_nope, v, k_rope = up[..., :128], up[..., 128:256], rows[:, 512:576]
    qo, ko = [0], [0]
    for n, m in lens:
        qo.append(qo[-1] + n)
        ko.append(ko[-1] + m)
    return q, k_nope, k_rope, v, i32(qo), i32(ko)


def reference(q, k_nope, k_rope, v, qo, ko, scale=SCALE, causal=True):
    heads, group = q.shape[1], q.shape[1] // v.shape[1]
    out = torch.zeros(*q.shape[:2], 128, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    mean = torch.zeros_like(out)
    qo, ko = qo.tolist(), ko.tolist()
    for b in range(len(qo) - 1):
        n, m = qo[b + 1] - qo[b], ko[b + 1] - ko[b]
        if n <= 0 or m <= 0:
            continue
        see = torch.arange(m, device="cuda") <= (m - n + torch.arange(n, device="cuda"))[:, None]
        rope = k_rope[ko[b]:ko[b + 1]].double()
        for h in range(heads):
            k = torch.cat([k_nope[ko[b]:ko[b + 1], h // group].double(), rope], 1)
            val = v[ko[b]:ko[b + 1], h // group].double()
            z = q[qo[b]:qo[b + 1], h].double() @ k.t() * scale
            if causal:
                z = z.masked_fill(~see, -math.inf)
            total = torch.logsumexp(z, -1)
            p = torch.exp(z - torch.where(torch.isfinite(total), total, 0.0)[:, None])
            out[qo[b]:qo[b + 1], h], mean[qo[b]:qo[b + 1], h] = p @ val, p @ val.abs()
            lse[qo[b]:qo[b + 1], h] = total / math.log(2.0)
    return out, lse, mean


def run(args, scale=SCALE, causal=True, flags=0, pad=0):
    q, batch = args[0], args[4].shape[0] - 1
    n, h = q.shape[:2]
    g_out, g_lse = Guarded(n * h * 256), Guarded(n * h * 4)
    g_out.body.fill_(0xA5)
    g_lse.body.fill_(0xA5)
    g_ws = Guarded(mla.prompt_attention_workspace_size(n, args[1].shape[0], h, batch))
    g_ws.body.fill_(0xFF)
    out, lse = mla.prompt_attention(*args, scale, is_causal=causal, out=g_out.view(torch.bfloat16, (n, h, 128)),
                                    lse=g_lse.view(torch.float32, (n, h)), workspace=g_ws.body)
    assert mla.device_status() == flags
    check_guards({"out": g_out, "lse": g_lse, "workspace": g_ws}, "prompt_attention")
    if pad:
        assert (out[n - pad:].view(torch.uint8) == 0xA5).all() and (lse[n - pad:].view(torch.uint8) == 0xA5).all()
    return out[:n - pad], lse[:n - pad]


def compare(args, what, scale=SCALE, causal=True, pad=0):
    want = reference(*args, scale=scale, causal=causal)
    n = args[0].shape[0] - pad
    check(*run(args, scale, causal, pad=pad), tuple(w[:n] for w in want), what)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 513, 1000])
@pytest.mark.parametrize("causal", [True, False])
def test_one_sequence(n, causal):
    compare(inputs(2, 2, [(n, n)], seed=n), f"{n}", causal=causal)


@pytest.mark.parametrize("n,m", [(1, 1), (1, 2), (1, 500), (3, 130), (64, 65), (100, 1000), (128, 384), (130, 129 + 256), (256, 2049),
                                 (300, 4), (300, 200), (257, 1), (129, 128), (5, 0), (0, 5), (600, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_queries_and_keys(n, m, causal):
    # context before the queries; fewer keys than queries: rows without keys
    compare(inputs(3, 1, [(n, m), (4, 9)], seed=n + m), f"{n} {m}", causal=causal)


@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (3, 3), (16, 16), (16, 4), (8, 1), (20, 5), (128, 128)])
def test_heads(h_q, h_kv):
    compare(inputs(h_q, h_kv, [(70, 70), (200, 330), (1, 40)], seed=h_q + h_kv), f"{h_q} {h_kv}")


@pytest.mark.parametrize("n,m", [(1, 700), (1, 5000), (7, 9001), (100, 513), (200, 2000), (300, 4000), (256, 20000)])
@pytest.mark.parametrize("heads", [1, 16, 60])
@pytest.mark.parametrize("causal", [True, False])
def test_few_rows_behind_many_keys(n, m, heads, causal):
    # an item's keys shared out over several CTAs, whose results are merged
    compare(inputs(heads, 1, [(n, m), (0, 3), (2, 300)], seed=n + m), f"{n} {m} {heads}", causal=causal)


@pytest.mark.parametrize("gap", [0, 8, 64])
@pytest.mark.parametrize("pad", [0, 1, 40])
def test_ragged_batches(gap, pad):
    lens = [(0, 0), (5, 5), (300, 300), (0, 70), (129, 500), (1, 1), (64, 64), (17, 3), (256, 257), (2, 900), (0, 0)]
    compare(inputs(4, 2, lens, seed=gap + pad, pad=pad, gap=gap), f"gap {gap} pad {pad}", pad=pad)


@pytest.mark.parametrize("n", [200, 1500, 5000])
def test_many_sequences(n):
    g = torch.Generator().manual_seed(n)
    lens = [(int(a), int(a + b)) for a, b in torch.randint(0, 30, (n, 2), generator=g).tolist()]
    compare(inputs(2, 2, lens, seed=n), f"{n} sequences")


@pytest.mark.parametrize("causal", [True, False])
def test_items_without_keys_among_others(causal):
    # several items per CTA, some of no tiles at all, some with tiles in one half alone
    lens = [(130, 0), (1, 1), (257, 900), (0, 50), (300, 2), (256, 0), (100, 400)] * 12
    compare(inputs(8, 4, lens, seed=15), "items without keys", causal=causal)


@pytest.mark.parametrize("heads,lens", [(1, [(5, 4000)]), (16, [(300, 500)] * 20)])
def test_negative_scales_of_long_and_of_many_items(heads, lens):
    compare(inputs(heads, 1, lens, seed=16), f"{heads} heads, scale -0.1", scale=-0.1)


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0, 1e-4])
def test_scales(scale):
    # 3.0: scores of hundreds, one key takes all of a row; negative: the smallest product is the largest score
    compare(inputs(2, 2, [(300, 300), (10, 600)], seed=3), f"scale {scale}", scale=scale)


@pytest.mark.parametrize("spread", [1e-3, 30.0])
def test_magnitudes(spread):
    args = inputs(2, 1, [(200, 400)], seed=4, spread=spread)
    out, lse, mean = reference(*args)
    got, got_lse = run(args)
    # scores of up to 900 * 192 / 14: fp32 products of 2^-24 of the sum of their absolute values, 2^-9 at most
    assert ((got.double() - out).abs() <= (2.0 ** -7) * mean + 2.0 ** -8 * out.abs() + 1e-30).all()
    assert ((got_lse.double() - lse).abs() <= 2.0 ** -7).all()


def test_rising_scores():
    # every tile's scores pass the last one's: O is rescaled at each
    args = inputs(2, 2, [(200, 1400)], seed=5)
    args[1].copy_((args[1].float() * torch.linspace(0.01, 6.0, 1400, device="cuda")[:, None, None]).to(torch.bfloat16))
    out, lse, mean = reference(*args)
    got, got_lse = run(args)
    assert ((got.double() - out).abs() <= (2.0 ** -8 + 2.0 ** -9) * mean + 2.0 ** -8 * out.abs()).all()
    assert ((got_lse.double() - lse).abs() <= 2.0 ** -9).all()


def test_what_other_sequences_hold_does_not_matter():
    args = inputs(2, 2, [(70, 70), (50, 130), (300, 333)], seed=6)
    want = run(args)
    q, k_nope, k_rope, v, qo, ko = args
    for bad in (float("nan"), float("inf"), -float("inf")):
        k2, r2, v2, q2 = k_nope.clone(), k_rope.clone(), v.clone(), q.clone()
        for t in (k2, r2, v2):
            t[70:200] = bad  # the second sequence
        q2[70:120] = bad
        got = run((q2, k2, r2, v2, qo, ko))
        for a, b in zip(got, want):
            assert torch.equal(a[:70], b[:70]) and torch.equal(a[120:], b[120:])
    # a key that no row sees yet: rows before it in other blocks
    v2 = v.clone()
    v2[70 + 129] = float("nan")  # last key of the second sequence: its last row alone sees it
    got = run((q, k_nope, k_rope, v2, qo, ko))
    assert torch.isnan(got[0][119]).all() and torch.isfinite(got[0][:70]).all() and torch.isfinite(got[0][120:]).all()


def test_rows_that_are_not_finite_stay_alone():
    args = inputs(2, 2, [(200, 200)], seed=7)
    want = run(args)
    args[0][50, 1, 3] = float("nan")
    out, lse = run(args)
    assert torch.isnan(out[50, 1]).all() and torch.isnan(lse[50, 1])
    keep = torch.ones(200, 2, dtype=torch.bool, device="cuda")
    keep[50, 1] = False
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


def test_repeated_runs_are_equal_and_a_graph_replays():
    args = inputs(8, 4, [(300, 700), (1, 3000), (513, 513), (40, 40)], seed=8)
    want = run(args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = mla.prompt_attention(*args, SCALE)
    for _ in range(20):
        got = run(args)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        out.zero_()
        graph.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    # new offsets in the same graph
    args[4].copy_(i32([0, 854, 854, 854, 854]))
    args[5].copy_(i32([0, 4253, 4253, 4253, 4253]))
    graph.replay()
    check(out, lse, reference(*args), "other offsets")
    assert mla.device_status() == 0


def test_repeated_calls_are_equal():
    # short and long items, several thousand: no field of one may be the next one's
    g = torch.Generator().manual_seed(3)
    lens = [(int(n), int(n + c)) for n, c in torch.randint(1, 400, (300, 2), generator=g).tolist()] + [(1500, 1500)]
    args = inputs(16, 16, lens, seed=14)
    want = mla.prompt_attention(*args, SCALE)
    for _ in range(100):
        got = mla.prompt_attention(*args, SCALE)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert mla.device_status() == 0


def test_bad_offsets_are_flagged_or_cut_off():
    q, k_nope, k_rope, v, _, _ = inputs(2, 2, [(100, 100)], seed=9)
    # past the rows: cut off there
    got = run((q, k_nope, k_rope, v, i32([0, 100 + 7]), i32([0, 100 + 7])))
    want = run((q, k_nope, k_rope, v, i32([0, 100]), i32([0, 100])))
    assert torch.equal(got[0], want[0])
    # decreasing: more blocks than 100 rows of 4 sequences have
    big = inputs(1, 1, [(2000, 2000)], seed=9)[:4]
    run((*big, i32([0, 2000, 0, 2000, 0, 2000]), i32([0, 2000, 0, 2000, 0, 2000])), flags=mla.DEVICE_BAD_SCHEDULE)


@pytest.mark.parametrize("stream_arg", [False, True])
def test_other_streams(stream_arg):
    args = inputs(4, 4, [(500, 500)], seed=10)
    want = run(args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    if stream_arg:
        out, lse = mla.prompt_attention(*args, SCALE, stream=s)
    else:
        with torch.cuda.stream(s):
            out, lse = mla.prompt_attention(*args, SCALE)
    s.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_empty_calls():
    q, k_nope, k_rope, v, qo, ko = inputs(2, 2, [(10, 10)], seed=11)
    out, lse = mla.prompt_attention(q[:0], k_nope, k_rope, v, i32([0, 0]), ko, SCALE)
    assert out.shape == (0, 2, 128) and lse.shape == (0, 2)
    out, lse = mla.prompt_attention(q, k_nope[:0], k_rope[:0], v[:0], qo, i32([0, 0]), SCALE)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert mla.device_status() == 0


def test_workspaces_are_checked():
    args = inputs(1, 1, [(20, 3000)], seed=13)  # (5 CTAs share the one item's keys)
    need = mla.prompt_attention_workspace_size(20, 3000, 1, 1)
    assert need > 5 * 256 * 129 * 4
    for ws in (torch.empty(need - 1, dtype=torch.uint8, device="cuda"), torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:]):
        with pytest.raises(ValueError, match="workspace"):
            mla.prompt_attention(*args, SCALE, workspace=ws)
    with pytest.raises(ValueError, match="k_rope must be"):
        mla.prompt_attention(args[0], args[1], args[2][:, :32], *args[3:], SCALE)
    with pytest.raises(ValueError, match="multiple of h_kv"):
        mla.prompt_attention(args[0].expand(-1, 3, -1).contiguous(), args[1].expand(-1, 2, -1).contiguous(), args[2],
                             args[3].expand(-1, 2, -1).contiguous(), *args[4:], SCALE)
    with pytest.raises(ValueError, match="positive multiple of 8"):
        mla.prompt_attention(args[0].expand(-1, 2, -1).contiguous(), args[1].expand(-1, 2, -1), args[2],
                             args[3].expand(-1, 2, -1), *args[4:], SCALE)


@pytest.mark.parametrize("heads", [2, 128])  # (one item a CTA; items from a list)
def test_watchdog_reports_an_expired_wait(heads):
    args = inputs(heads, 2, [(300, 300)], seed=12)
    from gpu_helpers import env
    with env(MLA_WATCHDOG_NS=20_000_000), overrides(debug_stall=True):
        mla.prompt_attention(*args, SCALE)
        torch.cuda.synchronize()
    assert mla.device_status() == mla.DEVICE_TIMEOUT
    compare(args, "after a timeout")
