"""Prompt attention over offsets that decrease: more blocks of query rows than the call has room for."""
import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from gpu_helpers import Guarded
from paged_reference import i32
from test_gpu_prompt import SCALE, inputs, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,keys", [(1, 2000), (32, 2000), (1, 6000)])  # an item a CTA; a plan; runs of items' keys
def test_more_blocks_than_the_call_has_room_for(heads, keys):
    # 2000 rows of 5 sequences are 12 blocks at most; these offsets name 24
    args = inputs(heads, 1, [(2000, keys)], seed=9)[:4]
    off = i32([0, 2000, 0, 2000, 0, 2000])
    run((*args, off, off.clamp(max=keys)), flags=mla.DEVICE_BAD_SCHEDULE)
    whole = i32([0, 2000, 2000, 2000, 2000, 2000])  # and the next call is as ever
    keep = i32([0, keys, keys, keys, keys, keys])
    a, b = run((*args, whole, keep)), run((*args, whole, keep))
    assert torch.isfinite(a[0]).all() and torch.equal(a[0], b[0])


def test_more_blocks_than_32_bits_hold():
    # 8192 sequences of 2^26 rows (which overlap in memory: 17 GB of results, none of them written) and as many
    # of none: 2^31 blocks
    n, batch = 1 << 26, 16384
    q = torch.zeros(n * 8 + 192, device="cuda", dtype=torch.bfloat16).as_strided((n, 1, 192), (8, 192, 1))
    k = torch.zeros(4, 1, 128, device="cuda", dtype=torch.bfloat16)
    rope = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    out = torch.empty(n, 1, 128, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(n, 1, device="cuda")
    off = i32([0, n]).repeat(batch // 2 + 1)[:batch + 1].contiguous()
    ws = Guarded(mla.prompt_attention_workspace_size(n, 4, 1, batch))
    mla.prompt_attention(q, k, rope, k, off, torch.zeros_like(off), SCALE, out=out, lse=lse, workspace=ws.body)
    assert mla.device_status() == mla.DEVICE_BAD_SCHEDULE
    ws.check("workspace")
