"""Token log probabilities in 64 bits, with bounds, for the tests."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def order(z):
    """Entries of every row, the largest first, the lowest index first among equals, NaN before all."""
    bits = (z.float() + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))
    key = torch.where(torch.isnan(z), 1 << 40, key)
    return torch.sort(key, dim=1, descending=True, stable=True).indices


def reference(logits, tokens, T, top=0, u=None, v=None):
    """{name: (value, bound)} in float64; top_index: whole numbers."""
    R, V = logits.shape
    T = float(torch.tensor(T, dtype=torch.float32))   # the library takes the temperature as a float32
    raw = logits.double()
    m = raw.amax(1, keepdim=True)
    empty = (m == -math.inf)
    pivot = torch.where(empty, 0.0, m)
    d = (raw - pivot) / T
    e = torch.exp(d)
    S = e.sum(1, keepdim=True)
    L = torch.log(S)
    p = torch.where(empty, 0.0, e / S)
    ds = torch.where(p > 0, d, 0.0)
    logp = torch.where(empty, -math.inf, d - L)
    H = -torch.where(p > 0, p * logp, 0.0).sum(1, keepdim=True)
    # FP32: an exponent d is off by the rounding of the difference, of log2(e) / T
    # and of the product (3 half steps of |d|, 1 more for the change of base),
    # 2^x by 2, a sum by its longest chain of additions (a thread's values of
    # a row, and the joins).
    n = 64 + V / 256
    D1, D2 = (p * ds.abs()).sum(1, keepdim=True), (p * ds * ds).sum(1, keepdim=True)
    S_rel = U32 * (4 * D1 + 4 + n)
    bL = S_rel + 2 * U32 * L.abs().nan_to_num(posinf=0.0)
    bL = torch.where(empty, 0.0, bL)
    bH = bL + U32 * (4 * D2 + (n + 8) * D1) + D1 * S_rel + U32 * (H.abs() + L.abs().nan_to_num(posinf=0.0))
    blp = 4 * U32 * torch.where(torch.isfinite(d), d.abs(), 0.0) + bL
    out = {"entropy": (H[:, 0], bH[:, 0]),
           "norm": (torch.cat((m, L), 1), torch.cat((torch.zeros_like(m), bL), 1))}
    has = (tokens >= 0) & (tokens < V)
    at = torch.where(has, tokens, 0).long()[:, None]
    out["logprob"] = (torch.where(has, logp.gather(1, at)[:, 0], 0.0), blp.gather(1, at)[:, 0])
    if top:
        best = order(logits)[:, :top]
        out["top_index"] = best.to(torch.int32)
        out["top_logprob"] = (logp.gather(1, best), blp.gather(1, best))
    if u is not None or v is not None:
        zero = torch.zeros(R, device=logits.device, dtype=torch.float64)
        u = zero if u is None else u.double()
        v = zero if v is None else v.double()
        off = ((u == 0) & (v == 0))[:, None] | empty | (~has & (v == 0))[:, None]
        take = torch.where(has, u, 0.0)[:, None]
        lp = torch.where(p > 0, logp, 0.0)
        grad = -p * (take + v[:, None] * (lp + H))
        size = take.abs() + v.abs()[:, None] * (lp.abs() + H.abs())
        bound = p * ((blp + 8 * U32) * size + v.abs()[:, None] * (blp + bH) + 8 * U32 * size)
        grad.scatter_add_(1, at, take)
        bound.scatter_add_(1, at, 4 * U32 * take.abs())
        # FP32 exponentials under 2^-126 become zero.
        bound = bound + 2.0 ** -120 * size
        out["grad"] = (torch.where(off, 0.0, grad / T), torch.where(off, 0.0, bound / T + 2.0 ** -126))
    return out


def close(got, pair, what=""):
    ref, bound = pair
    assert got.shape == ref.shape, what
    g = got.double()
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), what
    inf = torch.isinf(ref)
    assert torch.equal(g[inf], ref[inf]), what
    keep = torch.isfinite(ref)
    g, r, b = g[keep], ref[keep], bound[keep]
    assert torch.isfinite(g).all(), what
    allowed = b + HALF_STEP[got.dtype] * (r.abs() + b) + (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -149)
    worst = float(((g - r).abs() / allowed).max()) if g.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the allowed error"
