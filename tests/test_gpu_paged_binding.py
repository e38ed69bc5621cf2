"""The two ways through the binding of the paged-cache calls: the native one of the plain call and the
Python one (another stream, another form, refusals) launch the same work."""
import pytest
import torch

import paged_mla_decode_07_gb300 as mla
import test_gpu_prefix as prefix
import test_gpu_window as window
from paged_reference import i32

pytestmark = pytest.mark.gpu


def only_native(monkeypatch):
    monkeypatch.setattr(mla, "_launch", None)  # the Python way would call it


def current():
    return torch.cuda.current_stream()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_token"])
def test_window_decode_both_ways(monkeypatch, fmt):
    q, kv, sc, bt, L, _ = window.problem(fmt, 16, 2, (100, 700), 90, 5, seed=2)
    python = mla.window_decode(q, kv, bt, L, window.SCALE, 90, 5, kv_scales=sc, stream=current())
    # a Parameter is not a plain tensor
    python2 = mla.window_decode(torch.nn.Parameter(q, requires_grad=False), kv, bt, L, window.SCALE, 90, 5, kv_scales=sc)
    only_native(monkeypatch)
    native = mla.window_decode(q, kv, bt, L, window.SCALE, 90, 5, kv_scales=sc)
    out, lse = torch.empty_like(native[0]), torch.empty_like(native[1])
    given = mla.window_decode(q, kv, bt, L, window.SCALE, 90, 5, kv_scales=sc, out=out, lse=lse)
    assert given[0].data_ptr() == out.data_ptr() and given[1].data_ptr() == lse.data_ptr()
    for r in (python2, native, given):
        assert torch.equal(r[0], python[0]) and torch.equal(r[1], python[1])
        assert r[0].shape == (2, 2, 16, 512) and r[1].shape == (2, 2, 16)
    assert mla.device_status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_shared_prefix_decode_both_ways(monkeypatch, fmt):
    q, kv, sc, pt, plen, bt, lens, _ = prefix.problem(fmt, 16, 2, 300, (40, 90), True, seed=2)
    python = mla.shared_prefix_decode(q, kv, pt, plen, bt, lens, prefix.SCALE, is_causal=True, kv_scales=sc, stream=current())
    only_native(monkeypatch)
    native = mla.shared_prefix_decode(q, kv, pt, plen, bt, lens, prefix.SCALE, is_causal=True, kv_scales=sc)
    other = mla.shared_prefix_decode(q, kv, pt, plen, bt, lens, prefix.SCALE, is_causal=False, kv_scales=sc)
    assert torch.equal(native[0], python[0]) and torch.equal(native[1], python[1])
    assert not torch.equal(other[1], python[1])
    assert mla.device_status() == 0


def test_pages_and_store_both_ways(monkeypatch):
    old, new, free, cur = i32([5, 64, 0]), i32([3, 1, 70]), i32(range(20, 30)), i32([2])
    tab = torch.full((3, 4), 7, dtype=torch.int32, device="cuda")
    tab2 = tab.clone()
    python = mla.assign_pages(old, new, free, cur, tab, 80, stream=current())
    x = torch.randn(80, 576, device="cuda").to(torch.bfloat16)
    kv, kv2 = (torch.zeros(40, 64, 1, 656, dtype=torch.uint8, device="cuda") for _ in range(2))
    mla.cache_store(x[:, :512], x[:, 512:], python[2], kv, stream=current())
    only_native(monkeypatch)
    native = mla.assign_pages(old, new, free, cur, tab2, 80)
    mla.cache_store(x[:, :512], x[:, 512:], native[2], kv2)
    assert all(torch.equal(a, b) for a, b in zip(python, native)) and torch.equal(tab, tab2) and torch.equal(kv, kv2)
    assert mla.device_status() == 0


def test_refusals_name_the_argument():
    q, kv, sc, bt, L, _ = window.problem("bf16", 16, 1, (100, 700), 90, 5, seed=2)
    good = (q, kv, bt, L, window.SCALE)
    for kw, what in ((dict(window=0), "window"), (dict(window=5, sinks=-1), "sinks"), (dict(window=2 ** 31), "32 bits"),
                     (dict(window=2 ** 32 + 5), "32 bits"), (dict(window=5, out=q), "out"),
                     (dict(window=5, lse=L), "lse"), (dict(window=5, workspace=torch.empty(5, device="cuda")), "workspace"),
                     (dict(window=5, kv_scales=torch.ones(3, device="cuda")), "kv_scales")):
        with pytest.raises(ValueError, match=what):
            mla.window_decode(*good, **kw)
    for i, bad, what in ((0, q.float(), "q"), (0, q[..., :512], "q"), (0, q[:, :, ::2], "q"), (1, kv[:, :32], "kvcache"),
                         (1, kv.view(torch.uint8), "kvcache"), (2, bt.long(), "block_table"), (2, bt[:1], "batch rows"),
                         (3, L[:1], "batch rows"), (3, L.cpu(), "cache_seqlens"), (4, float("nan"), "sm_scale")):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError, match=what):
            mla.window_decode(*args, window=5)
    c, d, e, f = i32([1]), i32([1]), i32([4]), i32([0])
    t = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        mla.assign_pages(c, d, e, f, t, 1, cache_seqlens=d)
    with pytest.raises(ValueError, match="num_tokens"):
        mla.assign_pages(c, d, e, f, t, -1)
    with pytest.raises(ValueError, match="slot_map must have 4 entries"):
        mla.assign_pages(c, d, e, f, t, 4, slot_map=i32([1, 2]))
    lat, rope = torch.zeros(4, 512, device="cuda", dtype=torch.bfloat16), torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    slots = i32([0, 1, 2, 3])
    for args, what in (((lat[:3], rope, slots, kv), "rope"), ((lat, rope, slots[:3], kv), "slot_map"),
                       ((lat.t().contiguous().t(), rope, slots, kv), "contiguous"), ((lat, rope, slots, L), "kvcache"),
                       ((lat, torch.zeros(4, 65, device="cuda", dtype=torch.bfloat16)[:, :64], slots, kv), "rope_stride"),
                       ((lat, torch.zeros(4, 72, device="cuda", dtype=torch.bfloat16)[:, 1:65], slots, kv), "16-byte")):
        with pytest.raises(ValueError, match=what):
            mla.cache_store(*args)
    assert mla.device_status() == 0
