"""Bounded waits of the windowed and shared-prefix kernels: a wait that nothing completes runs out,
the call reports MLA_DEVICE_TIMEOUT, and the same context computes correct results afterwards."""
import pytest
import torch

import paged_mla_decode_07_gb300 as mla
import test_gpu_prefix as prefix
import test_gpu_window as window
from gpu_helpers import env, overrides
from paged_reference import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,h_q", [("bf16", 16), ("bf16", 128), ("fp8", 16), ("fp8_token", 16), ("fp8", 64)])
@pytest.mark.parametrize("lens", [(40, 900), (3000, 2500)])
def test_window_wait_runs_out(fmt, h_q, lens):
    q, kv, sc, bt, L, want = window.problem(fmt, h_q, 1, lens, 2000, 5, seed=1)
    with env(MLA_WATCHDOG_NS=200_000_000), overrides(debug_stall=True):
        mla.window_decode(q, kv, bt, L, window.SCALE, window=2000, sinks=5, kv_scales=sc)
        assert mla.device_status() & mla.DEVICE_TIMEOUT
    check(*window.run(q, kv, sc, bt, L, 2000, 5), want, f"{fmt} {h_q} after a timeout")


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_prefix_wait_runs_out(fmt):
    case = prefix.problem(fmt, 16, 1, 900, (40, 300), True, seed=1)
    q, kv, sc, pt, plen, bt, lens, want = case
    with env(MLA_WATCHDOG_NS=200_000_000), overrides(debug_stall=True):
        mla.shared_prefix_decode(q, kv, pt, plen, bt, lens, prefix.SCALE, kv_scales=sc)
        assert mla.device_status() & mla.DEVICE_TIMEOUT
    check(*prefix.run(*case[:7], True), want, f"{fmt} after a timeout")
