"""The sign of zero in FP8 cache writes: code = E4M3 of x / scale, so -0.0 is stored as 0x80 at every
scale, the same by slot and through the block table."""
import numpy as np
import pytest
import torch

import paged_mla_decode_07_gb300 as mla
from paged_reference import i32
from test_gpu_pages import run_store

pytestmark = pytest.mark.gpu


def tokens(n, power, seed):
    """Rows whose values are -0.0, +0.0 or below 2^power, with tiles and a token of zeros of both signs alone."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, 576, generator=g) * 2.0 ** power
    x[:, 1::3] = -0.0
    x[:, 2::7] = 0.0
    x[0, :128] = -0.0  # a tile
    if n > 1:
        x[1, :512] = -0.0  # a token
        x[1, ::5] = 0.0
    return x.to(torch.bfloat16).cuda()


@pytest.mark.parametrize("fmt", ["fp8", "fp8_token"])
@pytest.mark.parametrize("n", [1, 2, 33])
@pytest.mark.parametrize("power", [-100, -70, -20, 0, 12, 100])
def test_the_sign_of_zero_is_kept(fmt, n, power):
    x = tokens(n, power, seed=n + power + 200)
    slots = np.random.default_rng(n).permutation(64)[:n]
    run_store(x[:, :512], x[:, 512:], slots, 1, fmt)  # byte for byte, np.signbit of the quotients among them


@pytest.mark.parametrize("power", [-20, 0])
def test_both_stores_write_the_same_bytes(power):
    x = tokens(40, power, seed=5)
    a = torch.zeros(1, 64, 1, 656, dtype=torch.uint8, device="cuda")
    b = torch.zeros_like(a)
    mla.cache_store(x[:, :512], x[:, 512:], torch.arange(40, dtype=torch.int32, device="cuda"), a)
    mla.fp8_cache_store(x, i32([0, 40]), i32([0]), i32([[0]]), b)
    assert mla.device_status() == 0
    assert torch.equal(a, b)
