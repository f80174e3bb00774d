"""Distillation loss and gradient in 64 bits, with bounds, for the tests."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def reference(logits, teacher, index, weight, T):
    """(loss, lse, grad, bounds): float64. A row without a distribution on
    either side, or of weight 0, has loss 0 and gradient 0."""
    R, V = logits.shape
    # The library takes the temperature as a float32.
    T = float(torch.tensor(T, dtype=torch.float32))
    z = logits.double() / T
    idx = torch.where((index >= 0) & (index < V), index, V).long()
    t = torch.where(idx < V, teacher.double() / T, -math.inf)
    best = t.amax(1, keepdim=True)
    e = torch.exp(t - torch.where(best > -math.inf, best, 0.0))
    psum = e.sum(1, keepdim=True)
    # Everything relative to the row's largest logit: next to the lowest value
    # of a type the logarithm of the sum is lost even in 64 bits.
    top = z.amax(1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    lsum = torch.log(torch.exp(z - top).sum(1, keepdim=True))
    logq = (z - top) - lsum
    lse = (top + lsum)[:, 0]
    w = torch.ones(R, dtype=torch.float64, device=z.device) if weight is None else weight.double()
    on = (w != 0) & (psum[:, 0] > 0) & (lse > -math.inf)
    p = torch.where(on[:, None], e / psum, 0.0)
    lqj = logq.gather(1, idx.clamp(max=V - 1))
    term = torch.where(p > 0, p * (torch.log(p.clamp_min(1e-300)) - lqj), 0.0)
    loss = torch.where(on, w * T * T * term.sum(1), 0.0)
    wide = torch.zeros(R, V + 1, dtype=torch.float64, device=z.device)
    wide.scatter_add_(1, idx, p)
    q = torch.where(on[:, None], torch.exp(logq), 0.0)
    pv = wide[:, :V]
    f = torch.where(on, (w * T).abs(), 0.0)[:, None]
    grad = torch.where(on[:, None], (w * T)[:, None] * (q - pv), 0.0)
    # FP32: an exponent d is off by a few half steps of its size (the pivot
    # and the conversion to base 2: 4 half steps of |d|, 4 more of 2^x and
    # products), a sum of n values by n half steps at most; with a given lse
    # also by half a step of it.
    d = torch.where(torch.isfinite(logq), logq.abs(), 0.0)
    dm = d.amax(1, keepdim=True).clamp_min(1.0)
    n = 64 + V / 256   # longest chain of additions: a thread's values and the reduction
    qe = q * U32 * (4 * d + 2 * lse.abs()[:, None].nan_to_num(posinf=0.0) + 8 + n)
    td = torch.where(torch.isfinite(t), (t - torch.where(best > -math.inf, best, 0.0)).abs(), 0.0)
    pe = torch.where(p > 0, p * U32 * (4 * td + 16 + t.shape[1]), 0.0)
    wide.zero_().scatter_add_(1, idx, pe)
    bound_g = f * (qe + wide[:, :V] + 6 * U32 * (q + pv)) + 2.0 ** -126
    size = torch.where(p > 0, torch.log(p.clamp_min(1e-300)).abs() + torch.where(torch.isfinite(lqj), lqj.abs(), 0.0), 0.0)
    bound_l = torch.where(on, w.abs() * T * T * (
        (pe * size).sum(1) + (p * U32 * (8 * size + 8 * dm + n + 8 + t.shape[1])).sum(1)), 0.0)
    bound_s = torch.where(lse > -math.inf, U32 * (2 * lse.abs() + n + 8 + 4 * dm[:, 0]), 0.0)
    return (loss, bound_l), (lse, bound_s), (grad, bound_g)


def close(got, ref, bound, what=""):
    big = torch.finfo(got.dtype).max
    ref = torch.where(ref.abs() > big, torch.copysign(torch.full_like(ref, math.inf), ref), ref)   # as it rounds
    same = torch.isinf(ref) & (got.double() == ref)
    bound = torch.where(same, 0.0, bound)
    ref = torch.where(same, 0.0, ref)
    g = torch.where(same, 0.0, got.double())
    assert torch.isfinite(g).all(), what
    allowed = bound + HALF_STEP[got.dtype] * (ref.abs() + bound)
    if got.dtype == torch.float16:
        allowed = allowed + 2.0 ** -25
    worst = float(((g - ref).abs() / allowed.clamp_min(1e-300)).max()) if g.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the allowed error"
