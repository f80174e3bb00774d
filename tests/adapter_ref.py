"""Adapter projection and its gradients in 64 bits, with bounds on what the
library's FP32 sums and roundings may add, for the tests."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24                                             # half a step of FP32
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# T is kept as a 16-bit value and the 16-bit rounding of what it leaves, each
# off by at most half a step: 2^-9 of 2^-9 (bf16), 2^-12 of 2^-11 and the
# subnormal step below the row's largest value (f16); one bit more for safety
# of the scaling.
SPLIT = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -21}


def _rows(ids, n):
    for a in range(n):
        yield a, torch.nonzero(ids == a)[:, 0]


def forward(X, W, A, B, ids, scale, trans_w):
    """(Y, bound): float64 result and the error allowed to each FP32 element."""
    x, w = X.double(), (W.t() if trans_w else W).double()
    n, r, K = A.shape
    Y = x @ w
    mag = x.abs() @ w.abs()
    bound = (K + 2) * U32 * mag
    for a, m in _rows(ids, n):
        if not len(m):
            continue
        s = 1.0 if scale is None else float(scale[a])
        Aa, Ba = A[a].double(), B[a].double()
        t, tm = s * (x[m] @ Aa.t()), abs(s) * (x[m].abs() @ Aa.abs().t())
        Y[m] += t @ Ba
        off = (K + 3) * U32 * tm + SPLIT[X.dtype] * t.abs().amax(dim=1, keepdim=True)
        bound[m] += off @ Ba.abs() + (r + K + 4) * U32 * (tm @ Ba.abs() + mag[m])
    return Y, bound


def close(got, ref, bound, what=""):
    """Every element within its bound, and half a step of the result's own type."""
    allowed = bound + HALF_STEP[got.dtype] * (ref.abs() + bound)
    if got.dtype == torch.float16:
        allowed = allowed + 2.0 ** -25          # half a subnormal step
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), what
    worst = float((err / allowed.clamp_min(1e-300)).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the allowed error"


def backward(dY, X, W, A, B, ids, scale, trans_w):
    """((dX, bound), (dA, bound), (dB, bound))."""
    # dX is the forward form with W^T and the pair exchanged.
    dX = forward(dY, W, B, A, ids, scale, not trans_w)
    x, g = X.double(), dY.double()
    n, r, K = A.shape
    N = B.shape[2]
    z = lambda c: torch.zeros(n, r, c, dtype=torch.float64, device=X.device)  # noqa: E731
    dA, bA, dB, bB = z(K), z(K), z(N), z(N)
    for a, m in _rows(ids, n):
        if not len(m):
            continue
        s = 1.0 if scale is None else float(scale[a])
        for out, bnd, P, Q, left in ((dA, bA, B[a], x, g), (dB, bB, A[a], g, x)):
            P = P.double()
            t, tm = s * (left[m] @ P.t()), abs(s) * (left[m].abs() @ P.abs().t())
            out[a] = t.t() @ Q[m]
            off = (P.shape[1] + 3) * U32 * tm + SPLIT[X.dtype] * t.abs().max()
            bnd[a] = off.t() @ Q[m].abs() + (len(m) + 4) * U32 * 2 * (t.abs().t() @ Q[m].abs())
    return dX, (dA, bA), (dB, bB)
