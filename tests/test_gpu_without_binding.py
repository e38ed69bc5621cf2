"""The paged-cache calls through ctypes, in the forms that the native binding takes when it is there."""
import pytest
import torch

import paged_mla_decode_07_gb300 as mla
import test_gpu_prefix as prefix
import test_gpu_window as window
from paged_reference import i32

pytestmark = pytest.mark.gpu


class Subclass(torch.Tensor):
    """Not a plain tensor: the native binding leaves it to Python."""


@pytest.fixture
def no_binding(monkeypatch):
    mla.lib()
    monkeypatch.setattr(mla, "_native", None)


def count_launches(monkeypatch):
    n, launch = [], mla._launch
    monkeypatch.setattr(mla, "_launch", lambda *a: n.append(1) or launch(*a))
    return n


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_token"])
def test_window_decode(monkeypatch, fmt):
    q, kv, sc, bt, L, _ = window.problem(fmt, 16, 2, (100, 700), 90, 5, seed=2)
    native = mla.window_decode(q, kv, bt, L, window.SCALE, 90, 5, kv_scales=sc)
    n = count_launches(monkeypatch)
    sub = mla.window_decode(q.as_subclass(Subclass), kv, bt, L, window.SCALE, 90, 5, kv_scales=sc)
    assert len(n) == 1
    monkeypatch.setattr(mla, "_native", None)
    plain = mla.window_decode(q, kv, bt, L, window.SCALE, 90, 5, kv_scales=sc)
    assert len(n) == 2
    for r in (sub, plain):
        assert torch.equal(r[0], native[0]) and torch.equal(r[1], native[1])
    assert mla.device_status() == 0


def test_shared_prefix_decode(monkeypatch):
    q, kv, sc, pt, plen, bt, lens, _ = prefix.problem("fp8", 16, 2, 300, (40, 90), True, seed=2)
    args = (q, kv, pt, plen, bt, lens, prefix.SCALE, True)
    native = mla.shared_prefix_decode(*args, kv_scales=sc)
    n = count_launches(monkeypatch)
    monkeypatch.setattr(mla, "_native", None)
    plain = mla.shared_prefix_decode(*args, kv_scales=sc)
    assert len(n) == 1 and torch.equal(plain[0], native[0]) and torch.equal(plain[1], native[1])
    assert mla.device_status() == 0


def test_pages_and_store(no_binding):
    tab = torch.full((3, 4), 7, dtype=torch.int32, device="cuda")
    lens, off, slots, cur = mla.assign_pages(i32([5, 64, 0]), i32([3, 1, 70]), i32(range(20, 30)), i32([2]), tab, 80)
    assert lens.tolist() == [8, 65, 70] and off.tolist() == [0, 3, 4, 74] and int(cur[0]) == 5
    x = torch.randn(80, 576, device="cuda").to(torch.bfloat16)
    kv = torch.zeros(40, 64, 1, 576, dtype=torch.bfloat16, device="cuda")
    mla.cache_store(x[:, :512], x[:, 512:], slots, kv)
    assert torch.equal(kv.view(-1, 576)[slots[:74].long()], x[:74])
    assert mla.device_status() == 0
