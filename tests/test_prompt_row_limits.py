"""Row counts of prompt attention at which 32-bit roundings would wrap are refused (no GPU: before any
device is touched)."""
import ctypes

import pytest

import paged_mla_decode_07_gb300 as mla
from test_prompt_and_fp4_abi import PROMPT, lib, make  # noqa: F401 (the fixture)

MOST = 2 ** 31 - 512


@pytest.mark.parametrize("field", ["num_q", "num_k"])
@pytest.mark.parametrize("rows", [MOST + 1, 2 ** 31 - 1])
def test_rows_near_2_to_the_31(lib, field, rows):  # noqa: F811
    args = make(mla.PromptAttentionArgs, PROMPT, **{field: rows, "h_q": 1, "h_kv": 1})
    assert lib.mla_prompt_attention(args, None) == 2
    assert f"{field} = {rows} exceeds" in mla.last_error()
    n = ctypes.c_size_t()
    sizes = {"num_q": 10, "num_k": 10, **{field: rows}}
    assert lib.mla_prompt_attention_workspace_size(sizes["num_q"], sizes["num_k"], 1, 1, ctypes.byref(n)) == 2


def test_the_most_rows_pass_the_check(lib):  # noqa: F811
    n = ctypes.c_size_t()
    lib.mla_prompt_attention_workspace_size(MOST, MOST, 1, 1, ctypes.byref(n))
    assert "exceeds" not in mla.last_error()  # (without a GPU the call ends at the device, behind the checks)
