"""Host threads that make their first CUDA call through the library: no context is current there yet."""
import threading

import pytest
import torch

import paged_mla_decode_07_gb300 as mla
import test_gpu_prefix as prefix
import test_gpu_window as window
from paged_mla_decode_07_gb300 import workloads as W

pytestmark = pytest.mark.gpu


def in_a_thread(call):
    result = []

    def work():
        try:
            result.append(call())
        except Exception as e:  # noqa: BLE001 (told to the test's thread)
            result.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    if isinstance(result[0], Exception):
        raise result[0]
    return result[0]


def buffers(q, nbytes):
    return dict(out=torch.empty(*q.shape[:3], 512, dtype=torch.bfloat16, device="cuda"),
                lse=torch.empty(*q.shape[:3], device="cuda"), workspace=torch.empty(nbytes, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("fmt,h_q", [("bf16", 16), ("bf16", 64), ("bf16", 128), ("fp8", 16), ("fp8", 128)])
def test_window_decode(fmt, h_q):
    q, kv, sc, bt, L, _ = window.problem(fmt, h_q, 1, (100, 3000, 2900), 2000, 5, seed=2)
    call = lambda **kw: mla.window_decode(q, kv, bt, L, window.SCALE, 2000, 5, kv_scales=sc, **kw)
    want = call()
    kw = buffers(q, mla.window_decode_workspace_size(3, h_q=h_q, s_q=1, is_fp8=fmt != "bf16"))
    torch.cuda.synchronize()
    got = in_a_thread(lambda: call(**kw))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert mla.device_status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_shared_prefix_decode(fmt):
    q, kv, sc, pt, plen, bt, lens, _ = prefix.problem(fmt, 128, 1, 3000, (40, 90), True, seed=2)
    call = lambda **kw: mla.shared_prefix_decode(q, kv, pt, plen, bt, lens, prefix.SCALE, kv_scales=sc, **kw)
    want = call()
    kw = buffers(q, mla.shared_prefix_decode_workspace_size(2, h_q=128, s_q=1, prefix_table_len=pt.shape[0],
                                                            is_fp8=fmt != "bf16"))
    torch.cuda.synchronize()
    got = in_a_thread(lambda: call(**kw))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert mla.device_status() == 0


@pytest.mark.parametrize("name", ["tiny", "smoke_sparse", "smoke_pair_dense", "smoke_pair_sparse"])
def test_decode(name):
    if name == "tiny":
        inp = W.make_inputs("tiny")
    else:
        inp = W.make_inputs(W.custom(name=name, batch=2, h_q=128 if "pair" in name else 16, s_q=1,
                                     mode="dense" if name.endswith("dense") else "sparse", seqlens=(400, 90),
                                     **({} if name.endswith("dense") else {"topk": 128})), seed=6)
    w, d = inp.workload, inp.to("cuda")
    topk = 0 if d.indices is None else d.indices.shape[-1]
    fp8 = d.kvcache.dtype == torch.uint8
    sched, ns = mla.get_metadata(d.cache_seqlens, h_q=w.h_q, s_q=w.s_q, topk=topk, is_fp8=fp8)
    call = lambda **kw: mla.decode(d.q, d.kvcache, d.block_table, d.cache_seqlens, d.sm_scale, sched, ns,
                                   is_causal=w.causal, indices=d.indices, **kw)
    want = call()
    kw = buffers(d.q, max(256, mla.workspace_size(w.batch, h_q=w.h_q, s_q=w.s_q, topk=topk, is_fp8=fp8)))
    torch.cuda.synchronize()
    got = in_a_thread(lambda: call(**kw))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert mla.device_status() == 0
