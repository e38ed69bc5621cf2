"""Bounded waits of shared-prefix decode in blocks of 128 rows: the pair kernel over the prefix (and,
over bf16 rows, the own keys), the own-key kernel of an FP8 cache and the merge behind an expired wait."""
import pytest

import paged_mla_decode_07_gb300 as mla
import test_gpu_prefix as prefix
import test_gpu_window as window
from gpu_helpers import env, overrides
from paged_reference import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp8_token"])
@pytest.mark.parametrize("h_q", [16, 64, 128])
@pytest.mark.parametrize("length,own", [(900, (40, 300)), (0, (40, 0, 700)), (2000, (0, 0))])
def test_block_path_wait_runs_out(fmt, h_q, length, own):
    case = prefix.problem(fmt, h_q, 1, length, own, True, seed=h_q)
    q, kv, sc, pt, plen, bt, lens, want = case
    # (a forced part count: no clusters, so the blocks of 128 rows)
    with env(MLA_WATCHDOG_NS=100_000_000), overrides(num_parts=60, debug_stall=True):
        mla.shared_prefix_decode(q, kv, pt, plen, bt, lens, prefix.SCALE, is_causal=True, kv_scales=sc)
        assert mla.device_status() & mla.DEVICE_TIMEOUT
    with overrides(num_parts=60):
        check(*prefix.run(*case[:7], True), want, f"{fmt} {h_q} after a timeout, blocks")
    check(*prefix.run(*case[:7], True), want, f"{fmt} {h_q} after a timeout")


@pytest.mark.parametrize("fmt,h_q", [("bf16", 32), ("bf16", 128), ("fp8", 32), ("fp8_token", 128)])
def test_window_wait_runs_out_without_clusters(fmt, h_q):
    q, kv, sc, bt, L, want = window.problem(fmt, h_q, 1, (40, 900, 0), 2000, 5, seed=1)
    with env(MLA_WATCHDOG_NS=100_000_000), overrides(num_parts=60, debug_stall=True):
        mla.window_decode(q, kv, bt, L, window.SCALE, window=2000, sinks=5, kv_scales=sc)
        assert mla.device_status() & mla.DEVICE_TIMEOUT
    check(*window.run(q, kv, sc, bt, L, 2000, 5), want, f"{fmt} {h_q} after a timeout")
