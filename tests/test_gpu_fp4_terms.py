"""Decode over FP4 rows: what its 8-bit terms hold of the weights and of q, where one key has nearly all of a
row's weight and where a row of q has values far below its largest."""
import math

import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from fp4_reference import ROW, quantise, rows_of
from gpu_helpers import overrides
from paged_reference import i32

pytestmark = pytest.mark.gpu
PAGE, ALL = 64, 1 << 30


def cache(latent, rope):
    """A cache of the rows [n, 512] and [n, 64], n a multiple of 64, pages in order."""
    return rows_of(*quantise(latent), rope).view(-1, PAGE, 1, ROW).contiguous()


@pytest.mark.parametrize("h_q", [16, 32])
@pytest.mark.parametrize("pages", [512, 4096])
def test_many_small_weights_under_one_large_one(h_q, pages):
    """One key of weight 1, value 0, and n others of weight 2^-gap, value 1, all in one CTA: out is the others'
    share.  (The others share one physical page.)"""
    n = pages * PAGE - 1
    latent = torch.ones(2 * PAGE, 512, device="cuda", dtype=torch.bfloat16)
    rope = torch.zeros(2 * PAGE, 64, device="cuda", dtype=torch.bfloat16)
    latent[0], rope[0, 0] = 0.0, 1.0
    kv = cache(latent, rope)
    gaps = torch.tensor([12, 16, 18, 20, 22, 23, 24, 24.5, 25, 25.125, 25.25, 25.5, 26, 27, 28, 29], device="cuda")
    gaps = gaps.repeat(h_q // 16)
    q = torch.zeros(1, 1, h_q, 576, device="cuda", dtype=torch.bfloat16)
    q[0, 0, :, 512] = gaps  # (exact in bf16)
    table = i32([[0] + [1] * (pages - 1)])
    with overrides(num_parts=1):
        out, lse = mla.window_decode(q, kv, table, i32([n + 1]), math.log(2.0), window=ALL)
    assert mla.device_status() == 0
    w = torch.exp2(-gaps.double())
    total = 1 + n * w
    want = n * w / total
    # A weight is off by the larger of 2^-9 of itself and 2^-33 of the largest; the sums are fp32: n / 32 products
    # are added to O, each off by 2^-23 of it at most, 2^-10 in all; l likewise, by lanes, 2^-12; out is bf16, 2^-8.
    held = n * torch.maximum(w * 2.0 ** -9, torch.tensor(2.0 ** -33, device="cuda", dtype=torch.float64)) / total
    bound = held + want * (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -12)
    worst = ((out[0, 0].double() - want[:, None]).abs() / bound[:, None]).amax(1)
    assert (worst <= 1.0).all(), f"error by gap, of the bound: {worst.tolist()}"
    # (the scale's own rounding: 2^-23 of a gap)
    assert ((lse[0, 0].double() - (gaps.double() + torch.log2(total))).abs() <= 2.0 ** -12).all()


@pytest.mark.parametrize("h_q", [16, 32])
@pytest.mark.parametrize("size", [-40, 0, 30])
def test_queries_far_below_their_rows_largest(h_q, size):
    """A row of q whose largest value is a power of two that meets zeros, the others 2^-10 of it with their last
    bit set: one key's score is 511 times that value."""
    latent = torch.ones(PAGE, 512, device="cuda", dtype=torch.bfloat16)
    latent[:, 0] = 0.0
    kv = cache(latent, torch.zeros(PAGE, 64, device="cuda", dtype=torch.bfloat16))
    q = torch.zeros(1, 1, h_q, 576, device="cuda", dtype=torch.bfloat16)
    small = 2.0 ** size * torch.tensor([2.0 ** -e * (1 + odd * 2.0 ** -7) for e in (7, 8, 9, 10, 11, 12, 13, 14)
                                        for odd in (1, 127)], device="cuda", dtype=torch.float64)
    small = small.repeat(h_q // 16)
    q[0, 0, :, :512] = small[:, None].to(torch.bfloat16)
    q[0, 0, :, 0] = 2.0 ** size
    assert torch.equal(q[0, 0, :, 1].double(), small)
    scale = 2.0 ** -size
    out, lse = mla.window_decode(q, kv, i32([[0]]), i32([1]), scale, window=ALL)
    assert mla.device_status() == 0
    want = 511 * small * scale / math.log(2.0)
    # q is off by 2^-21 of its row's largest value, each of the 511 by as much; fp32 sums.  lse is made of the
    # score less 8 and of log2(2^8): a score of less than 4 is rounded to the step of numbers up to 8 in
    # the difference, 2^-21, by half of it at most, and lse is rounded from the two as far again: 2^-21 in all
    # (the row of 2^-14 * (1 + 127 / 128) has every one of its values off by the whole 2^-21, on one side).
    bound = 511 * 2.0 ** -21 / math.log(2.0) + 2.0 ** -20 * want + 2.0 ** -21
    assert ((lse[0, 0].double() - want).abs() <= bound).all(), ((lse[0, 0].double() - want).abs() / bound).tolist()
