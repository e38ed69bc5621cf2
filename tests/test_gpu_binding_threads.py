"""The native binding gives up the interpreter's lock while it allocates and launches."""
import sys
import threading
import time

import pytest
import torch

import paged_mla_decode_07_gb300 as mla
import test_gpu_prefix as prefix
import test_gpu_window as window
from paged_reference import i32

pytestmark = pytest.mark.gpu


def store():
    x = torch.randn(30000, 576, device="cuda").to(torch.bfloat16)
    kv = torch.zeros(500, 64, 1, 576, dtype=torch.bfloat16, device="cuda")
    args = (x[:, :512], x[:, 512:], torch.arange(30000, dtype=torch.int32, device="cuda"), kv, None)
    return "cache_store", args


def pages():
    batch = 4000
    args = (i32([9] * batch), i32([1] * batch), i32(range(batch)), i32([0]),
            torch.zeros(batch, 3, dtype=torch.int32, device="cuda"), batch, None,
            *(torch.empty(n, dtype=torch.int32, device="cuda") for n in (batch, batch + 1, batch, 1)))
    return "assign_pages", args


def outputs(q, nbytes):
    # all of them given: freeing a tensor gives up the lock too
    return (torch.empty(*q.shape[:3], 512, dtype=torch.bfloat16, device="cuda"), torch.empty(*q.shape[:3], device="cuda"),
            torch.empty(nbytes, dtype=torch.uint8, device="cuda"))


def windowed():
    q, kv, sc, bt, L, _ = window.problem("bf16", 64, 1, (1500,) * 8, 1000, 5, seed=2)
    return "window_decode", (q, kv, bt, L, window.SCALE, 1000, 5, sc,
                             *outputs(q, mla.window_decode_workspace_size(8, h_q=64, s_q=1, is_fp8=False)))


def prefixed():
    q, kv, sc, pt, plen, bt, lens, _ = prefix.problem("fp8", 128, 1, 1000, (40, 90, 5), True, seed=2)
    return "shared_prefix_decode", (q, kv, pt, plen, bt, lens, prefix.SCALE, True, sc,
                                    *outputs(q, mla.shared_prefix_decode_workspace_size(
                                        3, h_q=128, s_q=1, prefix_table_len=pt.shape[0], is_fp8=True)))


@pytest.mark.parametrize("make", [store, pages, windowed, prefixed])
def test_other_threads_run_meanwhile(make):
    """The interpreter is told to leave the lock with its thread for a minute unless it is given up.
    Calls fill the launch queue, so they wait in it; another thread must get its turn meanwhile."""
    name, args = make()
    mla.lib()
    call = getattr(mla._native, name)
    assert call(*args) is not None  # (the native way takes it)
    torch.cuda.synchronize()
    go, ran = threading.Lock(), []
    go.acquire()
    ready = threading.Event()

    def other():
        ready.set()
        with go:
            ran.append(True)

    t = threading.Thread(target=other)
    t.start()
    ready.wait()
    time.sleep(0.05)  # (it waits for `go`)
    interval = sys.getswitchinterval()
    sys.setswitchinterval(60)
    try:
        go.release()
        end = time.perf_counter() + 5
        while not ran and time.perf_counter() < end:
            call(*args)
        during = bool(ran)
    finally:
        sys.setswitchinterval(interval)
    t.join()
    torch.cuda.synchronize()
    assert during
    assert mla.device_status() == 0


def test_results_of_threads_that_call_at_once():
    cases = [windowed(), windowed(), prefixed(), prefixed()]
    want = [getattr(mla._native, n)(*a) for n, a in cases]
    torch.cuda.synchronize()
    got, errors = [[] for _ in cases], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()) as _:
                for _ in range(50):  # (outputs and workspaces of their own)
                    got[i].append(getattr(mla._native, cases[i][0])(*cases[i][1][:-3], None, None, None))
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 (told to the test's thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]
    for i, rows in enumerate(got):
        assert len(rows) == 50 and all(torch.equal(o, want[i][0]) and torch.equal(z, want[i][1]) for o, z in rows)
    assert mla.device_status() == 0
