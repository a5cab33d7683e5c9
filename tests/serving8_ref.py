"""The 8-bit cache's rules in plain torch on the CPU, exactly."""

import math

import torch

E4M3 = torch.float8_e4m3fn


def quantise(x):
    """Rows x [..., D] of bf16 or fp16 -> (values that the codes stand for before their scale, fp64; exponents' bytes).

    e4m3 has four bits of a value and no step below 2^-9; what is above 448 saturates."""
    x = x.double()
    top = x.abs().amax(-1)
    fine = torch.isfinite(top)
    m, e = torch.frexp(torch.where(fine, top, torch.zeros_like(top)))  # top = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = e - 9 + (m > 0.875).int()
    e = torch.where(top == 0, torch.full_like(e, -40), e.clamp(-40, 40))
    y = torch.ldexp(torch.where(fine[..., None], x, torch.zeros_like(x)), -e[..., None])
    _, size = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), size.clamp(min=-5) - 4)
    codes = (torch.round(y / step) * step).clamp(-448, 448)  # (torch.round: ties to even)
    return codes, torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)


def values(codes, exps):
    """What codes (e4m3, or the values that they stand for) and exponents stand for, in 64 bits."""
    scale = torch.ldexp(torch.ones(exps.shape, dtype=torch.float64), exps.int() - 127)
    scale = torch.where(exps == 255, torch.full_like(scale, math.nan), scale)
    return codes.double() * scale[..., None]
