"""MXFP4 tensors and their products in 64 bits, for the tests."""
from __future__ import annotations

import torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def quantize(x):
    """(codes [R, K'], scale codes [R, K' / 32]) of x's rows, one code a
    value, K' whole blocks. Every code is the one whose interval the value
    lies in; the ends of an interval belong to the even code."""
    R, K = x.shape
    wide = torch.zeros(R, (K + 31) // 32 * 32, dtype=torch.float64, device=x.device)
    wide[:, :K] = x.double()
    wide = wide.reshape(R, -1, 32)
    bad = ~torch.isfinite(wide).all(2, keepdim=True)
    wide = torch.where(bad, 0.0, wide)
    best = wide.abs().amax(2, keepdim=True)
    # frexp: best = m 2^e with 0.5 <= m < 1, so floor(log2(best)) = e - 1.
    s = torch.where(best > 0, torch.frexp(best)[1] - 3, -127).clamp(min=-127)
    y = wide.abs() / torch.exp2(s.double())
    code = torch.zeros_like(y, dtype=torch.uint8)
    for c in range(1, 8):
        middle = (GRID[c - 1] + GRID[c]) / 2
        code += (y > middle if c % 2 else y >= middle).to(torch.uint8)
    code += torch.signbit(wide).to(torch.uint8) * 8
    code = torch.where(bad, 0, code)
    scale = torch.where(bad, 255, s + 127).to(torch.uint8)
    return code.reshape(R, -1), scale[:, :, 0]


def pack(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()


def unpack(codes):
    return torch.stack((codes & 15, codes >> 4), 2).reshape(codes.shape[0], -1)


def values(code, scale, K):
    """What unpacked codes stand for, float64 [R, K]."""
    table = torch.tensor(GRID + tuple(-g for g in GRID), dtype=torch.float64, device=code.device)
    s = torch.exp2(scale.double() - 127)
    s = torch.where(scale == 255, torch.nan, s)
    return (table[code.long()].reshape(code.shape[0], -1, 32) * s[:, :, None]).reshape(code.shape[0], -1)[:, :K]


def close(got, ref, bound, what=""):
    """got's error is at most `bound` and the rounding to its own type."""
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    keep = ~torch.isnan(ref)
    g, r, b = got.double()[keep], ref[keep], bound[keep]
    allowed = b + HALF_STEP[got.dtype] * (r.abs() + b) + (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -126)
    worst = float(((g - r).abs() / allowed).max()) if g.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the allowed error"
