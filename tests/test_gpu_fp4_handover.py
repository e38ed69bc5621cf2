"""Decode over FP4 rows, repeated over tables in which pages and missing pages take turns: a page's state and
its rows belong together, whichever page takes its place in the copy ring."""
import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from fp4_reference import ROW
from test_gpu_fp4 import PAGE, SCALE, fp4_problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h_q,s_q", [(16, 1), (128, 1), (128, 2)])
@pytest.mark.parametrize("step", [2, 3])
def test_missing_pages_among_others(h_q, s_q, step):
    q, kv, _, bt, lens, _ = fp4_problem(h_q, s_q, [3000, 129, 1000, 4000, 64] * 8, 1 << 30, 0, seed=step)
    kv = kv.view(torch.uint8).view(-1, PAGE, 1, ROW)
    bt = bt.clone()
    bt[:, 1::step] = -1  # (pages 1, 1 + step, ..)

    def call():
        return mla.window_decode(q, kv, bt, lens, SCALE, window=1 << 30)

    want = call()
    assert torch.isfinite(want[0]).all() and torch.isfinite(want[1]).all()
    assert mla.device_status() == mla.DEVICE_BAD_PAGE
    # the keys of the pages that are there, as a cache of their own
    whole = [[p for p in row if p >= 0] for row in bt.tolist()]
    for b, length in ((2, 1000), (1, 129)):
        pages = whole[b][: len([j for j in range(-(-length // PAGE)) if j == 0 or (j - 1) % step])]
        rows = torch.cat([mla.cache_load(kv, torch.tensor([[p]], dtype=torch.int32, device="cuda"),
                                         torch.tensor([0, PAGE], dtype=torch.int32, device="cuda"), PAGE) for p in pages])
        keep = torch.tensor([p * PAGE + i < length for p in range(-(-length // PAGE)) if p == 0 or (p - 1) % step
                             for i in range(PAGE)], device="cuda")
        keys = rows[keep].double()
        last = length - 1 if s_q == 1 else length - 2  # (the first query token's position)
        at = torch.tensor([p * PAGE + i for p in range(-(-length // PAGE)) if p == 0 or (p - 1) % step
                           for i in range(PAGE)], device="cuda")[keep]
        keys = keys[at <= last]
        z = q[b, 0].double() @ keys.t() * SCALE
        w = torch.softmax(z, -1)
        mean = w @ keys[:, :512].abs()
        off = (want[0][b, 0].double() - w @ keys[:, :512]).abs()
        # P to 2^-9 and the scores' sums to 2^-9 of the mean, the result to 2^-8 (as the other tests have it)
        assert (off <= (2.0 ** -8 + 2.0 ** -9) * mean + 2.0 ** -8 * (w @ keys[:, :512]).abs()).all()
    for _ in range(200):
        out, lse = call()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert mla.device_status() == mla.DEVICE_BAD_PAGE
