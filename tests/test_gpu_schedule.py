"""Schedules of windowed decode with more problems than a CTA has threads: runs of problems per thread,
long stretches of elements without keys, parts that end inside them."""
import numpy as np
import pytest
import torch

from fp4_reference import Fp4Cache
from gpu_helpers import overrides
from paged_reference import check
from test_gpu_fp4 import run as run_fp4
from test_gpu_window import problem
from test_gpu_window import run as run_window

pytestmark = pytest.mark.gpu


def lengths(n, seed):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 150, n)
    for _ in range(6):  # elements without keys, more of them in a row than a thread has
        at = rng.integers(0, n)
        lens[at:at + rng.integers(2, n // 8)] = 0
    lens[rng.integers(0, n, 3)] = 1500
    lens[:rng.integers(0, 40)] = 0
    lens[n - rng.integers(1, 40):] = 0
    return tuple(int(x) for x in lens)


@pytest.mark.parametrize("fmt,h_q,n", [("bf16", 16, 1700), ("fp8_token", 16, 900), ("bf16", 64, 1000), ("fp8", 40, 1300),
                                       ("bf16", 128, 800), ("fp4", 16, 2000), ("fp4", 48, 1000)])
def test_more_problems_than_threads(fmt, h_q, n):
    make = {"make": Fp4Cache} if fmt == "fp4" else {}
    run = run_fp4 if fmt == "fp4" else run_window
    q, kv, sc, bt, L, want = problem(fmt, h_q, 1, lengths(n, n), 1000, 10, seed=n, **make)
    check(*run(q, kv, sc, bt, L, 1000, 10), want, f"{fmt} {h_q} heads, {n} elements")
    for parts in (1, 37, 1000):
        with overrides(num_parts=parts):
            check(*run(q, kv, sc, bt, L, 1000, 10), want, f"{fmt} {h_q} heads, {n} elements, {parts} parts")


@pytest.mark.parametrize("fmt,h_q", [("bf16", 16), ("fp4", 16)])
def test_no_keys_at_all(fmt, h_q):
    make = {"make": Fp4Cache} if fmt == "fp4" else {}
    run = run_fp4 if fmt == "fp4" else run_window
    q, kv, sc, bt, L, want = problem(fmt, h_q, 1, (0,) * 1000, 100, 1, seed=3, **make)
    out, lse = run(q, kv, sc, bt, L, 100, 1)
    assert not out.any() and torch.isneginf(lse).all()
