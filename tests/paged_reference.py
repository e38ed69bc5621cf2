"""Inputs and 64-bit references of the windowed and the shared-prefix decode tests."""
import math

import numpy as np
import torch

PAGE = 64
D_QK, D_V = 576, 512
ROW = {"bf16": 1152, "fp8": 656, "fp8_token": 640}


def i32(x):
    return torch.tensor(np.asarray(x, np.int64), dtype=torch.int32, device="cuda")


class Cache:
    """Logical key rows (float64 values and stored bytes) and the paged cache they are put into.
    Every slot that no key occupies holds NaNs."""

    def __init__(self, fmt, seed, pages):
        self.fmt, self.pages = fmt, pages
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.order = torch.randperm(pages, generator=self.g, device="cuda").tolist()
        self.used = 0
        self.raw = torch.full((pages * PAGE, ROW[fmt]), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every format
        self.scales = torch.full((pages * PAGE,), float("nan"), device="cuda") if fmt == "fp8_token" else None

    def rows(self, n):
        """n random key rows: (values float64 [n, 576], bytes [n, row], scales [n] or None)."""
        x = torch.randn(n, D_QK, generator=self.g, device="cuda")
        rope = x[:, D_V:].to(torch.bfloat16)
        if self.fmt == "bf16":
            v = x.to(torch.bfloat16)
            return v.double(), v.contiguous().view(torch.uint8), None
        t = x[:, :D_V].reshape(n, 4 if self.fmt == "fp8" else 1, -1)
        s = (t.abs().amax(-1, keepdim=True) / 448.0)
        codes = (t / s).to(torch.float8_e4m3fn)
        lat = (codes.float() * s).to(torch.bfloat16).double().reshape(n, D_V)
        parts = [codes.view(torch.uint8).reshape(n, D_V)]
        if self.fmt == "fp8":
            parts.append(s.reshape(n, 4).contiguous().view(torch.uint8))
        parts.append(rope.contiguous().view(torch.uint8))
        return torch.cat([lat, rope.double()], 1), torch.cat(parts, 1), s.reshape(n) if self.fmt == "fp8_token" else None

    def put(self, n, keep=None):
        """Place n keys; returns (values, page ids).  keep: positions that are stored; pages that hold
        none of them get the id -1 and the other positions NaNs."""
        values, raw, scales = self.rows(max(n, 1))
        keep = np.arange(n) if keep is None else np.asarray(sorted(keep), np.int64)
        ids = []
        for pg in range(-(-n // PAGE)):
            mine = keep[(keep >= pg * PAGE) & (keep < (pg + 1) * PAGE)]
            if len(mine) == 0:
                ids.append(-1)
                continue
            page = self.order[self.used]
            self.used += 1
            ids.append(page)
            src = torch.from_numpy(mine).cuda()
            dst = src - pg * PAGE + page * PAGE
            self.raw[dst] = raw[src]
            if scales is not None:
                self.scales[dst] = scales[src]
        return values[:n], ids

    def tensors(self):
        kv = self.raw.view(self.pages, PAGE, 1, -1)
        if self.fmt == "bf16":
            kv = kv.view(torch.bfloat16)
        return kv, self.scales.view(self.pages, PAGE) if self.scales is not None else None


def table(rows, fill=-1, width=None):
    width = max([1] + [len(r) for r in rows]) if width is None else width
    t = np.full((len(rows), width), fill)
    for b, r in enumerate(rows):
        t[b, :len(r)] = r
    return i32(t)


def attend(q, keys, scale):
    """One query token [h, 576] over keys [n, 576] (float64): (out, lse base 2, mean |v| under the softmax)."""
    h = q.shape[0]
    if keys.shape[0] == 0:
        z = torch.zeros(h, D_V, dtype=torch.float64, device=q.device)
        return z, torch.full((h,), -math.inf, dtype=torch.float64, device=q.device), z
    s = (q.double() @ keys.t()) * scale
    p = torch.softmax(s, -1)
    v = keys[:, :D_V]
    return p @ v, torch.logsumexp(s, -1) / math.log(2.0), p @ v.abs()


def check(out, lse, want, what):
    """out and lse against the 64-bit values.  Each probability is rounded to bf16 once (relative
    2^-8 at most) and so is the result; an FP8 value may enter its sum as code x scale, without the
    rounding to bf16 that its definition has, 2^-8 of |v| at most; an fp32 dot product of 576 terms whose absolute values sum to
    about 15 is off by at most 15 * 576 * 2^-24 = 2^-10.9, which enters a probability and the sum it
    is divided by: 2^-9.9 of the mean |v|, taken as 2^-9."""
    want_out, want_lse, mean_v = want
    out, lse = out.double(), lse.double()
    assert torch.isfinite(out).all(), f"{what}: non-finite output"
    value = 2.0 ** -8 if what.startswith("fp8") else 0.0
    bound = (2.0 ** -8 + 2.0 ** -9 + value) * mean_v + 2.0 ** -8 * want_out.abs() + 1e-30
    worst = ((out - want_out).abs() / bound).max().item() if out.numel() else 0.0
    assert worst <= 1.0, f"{what}: error is {worst:.3f} of the bound"
    fin = torch.isfinite(want_lse)
    assert torch.equal(torch.isfinite(lse), fin), f"{what}: rows without keys differ"
    assert torch.equal(lse[~fin], want_lse[~fin]), f"{what}: lse of rows without keys"
    if fin.any():
        assert (lse[fin] - want_lse[fin]).abs().max().item() <= 2.0 ** -9, f"{what}: lse"
