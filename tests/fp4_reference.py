"""FP4 cache rows in plain 64-bit arithmetic: quantisation, the row's bytes, and the values they stand for."""
import torch

from paged_reference import PAGE, Cache

ROW = 400
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def quantise(x):
    """(codes int64 [n, 512] of three bits, signs int64 [n, 512], exponents int64 [n, 16]) of latents [n, 512].
    Scale 2^e: the smallest with amax <= 6 * 2^e, -13 <= e <= 13; nearest code, ties to the even one."""
    t = x.double().reshape(-1, 16, 32)
    amax = t.abs().amax(-1)
    e = torch.full_like(amax, 13.0)
    for k in range(12, -14, -1):
        e = torch.where(amax <= 6.0 * 2.0 ** k, torch.full_like(e, float(k)), e)
    y = (t.abs() * torch.exp2(-e)[..., None]).clamp(max=6.0)
    d = (y[..., None] - GRID.to(x.device)).abs()
    odd = torch.tensor([0, 1] * 4, device=x.device) * 1e-9  # of two codes equally near the even one
    code = (d + odd).argmin(-1)
    return code.reshape(-1, 512), torch.signbit(t).long().reshape(-1, 512), e.long()


def rows_of(code, sign, e, rope):
    """The 400 bytes of each row; rope bf16 [n, 64]."""
    n = len(code)
    out = torch.zeros(n, ROW, dtype=torch.uint8, device=code.device)
    nib = code.reshape(n, 64, 8).clone()
    s = sign.reshape(n, 64, 8)
    for i in range(8):  # the sign of dim i is the top bit of nibble 2 i + 1, of dim 4 + i of nibble 2 i
        nib[:, :, 2 * i + 1 if i < 4 else 2 * (i - 4)] |= s[:, :, i] << 3
    out[:, :256] = (nib[:, :, 0::2] | (nib[:, :, 1::2] << 4)).reshape(n, 256).to(torch.uint8)
    out[:, 256:272] = (e + 127).to(torch.uint8)
    out[:, 272:] = rope.contiguous().view(torch.uint8)
    return out


def values_of(code, sign, e):
    v = GRID.to(code.device)[code] * (1 - 2 * sign)
    return (v.reshape(-1, 16, 32) * torch.exp2(e.double())[..., None]).reshape(-1, 512)


def stored(x):
    """Float64 values [n, 576] that rows written from bf16 [n, 576] stand for."""
    return torch.cat([values_of(*quantise(x[:, :512])), x[:, 512:].double()], 1)


class Fp4Cache(Cache):
    """Cache with FP4 rows; slots that no key occupies hold 0xFF bytes (NaN RoPE values, the largest codes)."""

    def __init__(self, fmt, seed, pages):
        super().__init__("bf16", seed, pages)
        self.fmt = fmt
        self.raw = torch.full((pages * PAGE, ROW), 0xFF, dtype=torch.uint8, device="cuda")

    def rows(self, n):
        x = torch.randn(n, 576, generator=self.g, device="cuda")
        x[:, :512] *= torch.rand(n, 1, generator=self.g, device="cuda") + 0.5
        x = x.to(torch.bfloat16)
        q = quantise(x[:, :512])
        return torch.cat([values_of(*q), x[:, 512:].double()], 1), rows_of(*q, x[:, 512:]), None
