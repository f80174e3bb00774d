"""Adapters of several users trained at once, by distillation from a teacher's
top logits, then served for single tokens.

A student's head W (hidden x vocabulary) is frozen; every user has a low-rank
pair of their own beside it. A batch holds rows of all users. One step:

    logits = X W + scale[a] (X A[a]^T) B[a]              adapter_gemm
    loss, d logits from the teacher's top entries        distill (in the logits' place)
    dA, dB of every user in one pass                     adapter_backward

The teacher here is the student's head plus a hidden low-rank change per user,
so the loss can fall far. Run: python examples/distill_adapters.py
"""
from __future__ import annotations

import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import shape_adaptive_matrix_amd as sam  # noqa: E402


def teacher_logits(X, W, change, ids):
    """What the teacher says: X (W + change of the row's user)."""
    low, high = change
    return sam.adapter_gemm(X, W, low, high, ids)


def train(users=3, hidden=256, vocabulary=2048, rank=8, rows=512, top=32, steps=60, rate=0.05, temperature=2.0, seed=0,
          dtype=torch.bfloat16):
    """Returns (W, A, B, scale, losses): the mean loss of a row, step by step."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, by):
        return torch.randn(*shape, device="cuda", generator=g) * by

    W = normal(hidden, vocabulary, by=hidden ** -0.5).to(dtype)
    change = normal(users, 4, hidden, by=hidden ** -0.5).to(dtype), normal(users, 4, vocabulary, by=1.0).to(dtype)
    # A starts at random values and B at zero, so that the student starts at W.
    A, B = normal(users, rank, hidden, by=hidden ** -0.5), torch.zeros(users, rank, vocabulary, device="cuda")
    scale = torch.ones(users, device="cuda")
    optimizer = torch.optim.Adam([A, B], lr=rate)
    losses = []
    for _ in range(steps):
        X = normal(rows, hidden, by=1.0).to(dtype)
        ids = torch.randint(0, users, (rows,), device="cuda", generator=g).sort().values.to(torch.int32)
        best = teacher_logits(X, W, change, ids).topk(top, dim=1)
        t, index = best.values.contiguous(), best.indices.to(torch.int32)
        weight = torch.full((rows,), 1.0 / rows, device="cuda")

        A16, B16 = A.to(dtype), B.to(dtype)
        logits = sam.adapter_gemm(X, W, A16, B16, ids, scale, out_dtype=dtype)
        loss, d_logits = sam.distill(logits, t, index, weight, temperature, grad=logits)
        _, A.grad, B.grad = sam.adapter_backward(d_logits, X, W, A16, B16, ids, scale, need_dx=False)
        optimizer.step()
        losses.append(loss.sum())
    return W, A.to(dtype), B.to(dtype), scale, torch.stack(losses).tolist()


def next_token_logits(x, W, A, B, scale, user):
    """One user's next token: x of one row."""
    ids = torch.tensor([user], dtype=torch.int32, device=x.device)
    return sam.adapter_gemm(x, W, A, B, ids, scale)


def main():
    W, A, B, scale, losses = train()
    print(f"loss of a row: {losses[0]:.3f} at the start, {losses[-1]:.3f} after {len(losses)} steps")
    x = torch.randn(1, W.shape[0], device="cuda").to(W.dtype)
    for user in range(A.shape[0]):
        print(f"user {user}: token {int(next_token_logits(x, W, A, B, scale, user).argmax())}")
    print(f"no adapter: token {int(next_token_logits(x, W, A, B, scale, -1).argmax())}")


if __name__ == "__main__":
    main()
