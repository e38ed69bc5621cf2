"""Calls from several host threads: kernels whose shared memory varies with the call are launched with
their own size, whatever other threads launch at the same time."""
import ctypes
import threading

import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from paged_mla_decode_07_gb300 import workloads as W
from paged_reference import i32

pytestmark = pytest.mark.gpu


def pages(batch):
    old = i32([(7 * i) % 200 for i in range(batch)])
    new, free, cur = i32([1] * batch), i32(range(batch)), i32([0])
    tab = torch.zeros(batch, 5, dtype=torch.int32, device="cuda")
    out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (batch, batch + 1, batch, 1)]
    a = mla.AssignPagesArgs(old.data_ptr(), new.data_ptr(), batch, free.data_ptr(), batch, cur.data_ptr(), tab.data_ptr(), 5,
                            mla.MAX_PAGES, batch, *(t.data_ptr() for t in out))
    return (old, new, free, cur, tab, a), out, lambda stream: mla.lib().mla_assign_pages(ctypes.byref(a), stream)


def metadata(batch):
    lens = i32([(37 * i) % 500 for i in range(batch)])
    out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in mla.metadata_size(batch, h_q=16, s_q=1, topk=0, is_fp8=False)]
    ptr = [ctypes.c_void_p(t.data_ptr()) for t in (lens, *out)]
    return lens, out, lambda stream: mla.lib().mla_get_metadata(ptr[0], batch, 16, 1, 0, 0, ptr[1], ptr[2], stream)


def index(topk):
    d = W.make_index_inputs(W.IndexWorkload("threads", batch=1, n_new=1, h_idx=8, topk=topk, seqlens=(300,)), seed=1)
    t = [x.cuda() for x in (d.q_codes, d.q_scales, d.weights, d.row_offsets, d.k_codes, d.k_scales, d.block_table,
                            d.cache_seqlens)]
    q, qs, w, off, k, ks, bt, lens = (x.data_ptr() for x in t)
    out = [torch.empty(1, topk, dtype=torch.int32, device="cuda")]
    ws = torch.empty(mla.index_topk_workspace_size(1, t[6].shape[1]), dtype=torch.uint8, device="cuda")
    a = mla.IndexTopkArgs()
    for f, v in dict(q_codes=q, q_scales=qs, weights=w, num_tokens=1, h_idx=8, row_offsets=off, batch=1, max_new_tokens=1,
                     k_codes=k, k_scales=ks, num_pages=t[4].shape[0], page_size=64, block_table=bt,
                     block_table_stride=t[6].shape[1], cache_seqlens=lens, relu=0, topk=topk, workspace=ws.data_ptr(),
                     workspace_bytes=ws.nbytes, indices=out[0].data_ptr()).items():
        setattr(a, f, v)
    return (t, ws, a), out, lambda stream: mla.lib().mla_index_topk(ctypes.byref(a), stream)


@pytest.mark.parametrize("make,large,small", [(pages, 16384, 4000), (metadata, 16384, 50), (index, 16384, 16)])
def test_two_threads_with_different_sizes(make, large, small):
    cases = [make(large), make(small)]
    want = []
    for _, out, call in cases:
        assert call(torch.cuda.current_stream().cuda_stream) == 0, mla.last_error()
        want.append([t.clone() for t in out])
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(2)

    def work(i):
        stream = torch.cuda.Stream()
        start.wait()
        for _ in range(20000):
            if errors:
                break
            if cases[i][2](stream.cuda_stream) != 0:
                errors.append(mla.last_error())
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]
    assert mla.device_status() == 0
    for (_, out, _), ref in zip(cases, want):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
