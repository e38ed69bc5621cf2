"""Dimensions that do not fit the C arguments' 32 bits are refused, not cut off."""
import pytest
import torch

import paged_mla_decode_07_gb300 as mla


@pytest.mark.parametrize("shape", [(2 ** 31,), (2 ** 32 + 4,), (1, 2 ** 31), (2 ** 32 + 1, 1)])
def test_checks_refuse_them(shape):
    t = torch.empty(shape, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        mla._need(t, "block_table", torch.int32, ndim=len(shape))
    mla._need(torch.empty(2 ** 31 - 1, dtype=torch.int32, device="meta"), "slot_map", torch.int32, ndim=1)


@pytest.mark.gpu
def test_a_free_list_of_more_entries():
    # 2^32 + 4 entries, of which the first six are wanted (cut off, four would be left)
    free = torch.empty(2 ** 32 + 4, dtype=torch.int32, device="cuda")
    free[:6] = torch.arange(6, dtype=torch.int32, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    table = torch.full((1, 8), -1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="32 bits"):
        mla.assign_pages(0 * one, 384 * one, free, 0 * one, table, 384)
    assert (table == -1).all()
