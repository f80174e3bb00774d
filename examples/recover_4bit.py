"""A model whose output head is kept in 4 bits, brought back by adapters.

The head (vocabulary x hidden) is rounded to MXFP4 once and frozen. Low-rank
adapters on the projection before it learn to make up for the rounding, from
the most likely entries of the 16-bit model or from sampled tokens. One step:

    h = X W + scale[a] (X A[a]^T) B[a]                   adapter_gemm
    logits = q(h) Hq^T                                   linear_mxfp4
    teacher: loss, d logits from its top entries         token_logprobs, distill
    tokens:  log probabilities, entropy, d logits        token_logprobs, token_logprobs_grad
    d h = d logits Hq                                    linear_mxfp4_backward
    dA, dB                                               adapter_backward

Run: python examples/recover_4bit.py
"""
from __future__ import annotations

import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import shape_adaptive_matrix_amd as sam  # noqa: E402


def model(hidden=256, vocabulary=2048, users=2, rank=8, seed=0, dtype=torch.bfloat16):
    """Weights of the 16-bit model, the 4-bit head and fresh adapters."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, by):
        return torch.randn(*shape, device="cuda", generator=g) * by

    W = normal(hidden, hidden, by=hidden ** -0.5).to(dtype)
    head = normal(hidden, vocabulary, by=2 * hidden ** -0.5).to(dtype)   # stored K x N
    codes, scales = sam.quantize_mxfp4(head, trans=True)
    A, B = normal(users, rank, hidden, by=hidden ** -0.5), torch.zeros(users, rank, hidden, device="cuda")
    return {"W": W, "head": head, "codes": codes, "scales": scales, "A": A, "B": B, "scale": torch.ones(users, device="cuda"),
            "g": g}


def forward(m, X, ids, dtype=torch.bfloat16):
    h = sam.adapter_gemm(X, m["W"], m["A"].to(dtype), m["B"].to(dtype), ids, m["scale"], out_dtype=dtype)
    return h, sam.linear_mxfp4(h, m["codes"], m["scales"], out_dtype=dtype)


def backward(m, X, ids, d_logits, dtype=torch.bfloat16):
    d_h = sam.linear_mxfp4_backward(d_logits, m["codes"], m["scales"], m["W"].shape[1], out_dtype=dtype)
    _, dA, dB = sam.adapter_backward(d_h, X, m["W"], m["A"].to(dtype), m["B"].to(dtype), ids, m["scale"], need_dx=False)
    return d_h, dA, dB


def teacher_entries(m, X, top, dtype=torch.bfloat16):
    """The 16-bit model's most likely entries of every row: log probabilities and indices."""
    logits = sam.gemm(sam.gemm(X, m["W"]).to(dtype), m["head"])
    none = torch.full((X.shape[0],), -1, dtype=torch.int32, device="cuda")
    return sam.token_logprobs(logits, none, top=top)[3:]


def step(m, X, ids, top=32, tokens=None, entropy_weight=0.01):
    """Loss of every row and what the step computed: towards the teacher's entries, or (tokens given) towards those
    tokens with a bonus for entropy."""
    rows = X.shape[0]
    h, logits = forward(m, X, ids)
    kept = logits.clone()
    if tokens is None:
        best, index = teacher_entries(m, X, top)
        weight = torch.full((rows,), 1.0 / rows, device="cuda")
        loss, d_logits = sam.distill(logits, best, index, weight, grad=logits)
        more = {"best": best, "index": index}
    else:
        logprob, entropy, norm = sam.token_logprobs(logits, tokens)
        u = torch.full((rows,), -1.0 / rows, device="cuda")
        loss = (-logprob - entropy_weight * entropy) / rows
        d_logits = sam.token_logprobs_grad(logits, tokens, norm, entropy, u, entropy_weight * u, grad=logits)
        more = {"logprob": logprob, "entropy": entropy, "norm": norm}
    d_h, dA, dB = backward(m, X, ids, d_logits)
    return {"loss": loss, "h": h, "logits": kept, "d_logits": d_logits, "d_h": d_h, "dA": dA, "dB": dB, **more}


def train(steps=60, rows=512, rate=0.02, objective="teacher", seed=0, **sizes):
    m = model(seed=seed, **sizes)
    optimizer = torch.optim.Adam([m["A"], m["B"]], lr=rate)
    users, hidden = m["A"].shape[0], m["W"].shape[0]
    losses = []
    for _ in range(steps):
        X = torch.randn(rows, hidden, device="cuda", generator=m["g"]).to(m["W"].dtype)
        ids = torch.randint(0, users, (rows,), device="cuda", generator=m["g"]).sort().values.to(torch.int32)
        tokens = teacher_entries(m, X, 1)[1][:, 0].contiguous() if objective == "tokens" else None
        s = step(m, X, ids, tokens=tokens)
        m["A"].grad, m["B"].grad = s["dA"], s["dB"]
        optimizer.step()
        losses.append(s["loss"].sum())
    return m, torch.stack(losses).tolist()


def next_token(m, x, user, top=5):
    """The most likely next tokens of one row, with their log probabilities and the row's entropy."""
    ids = torch.tensor([user], dtype=torch.int32, device="cuda")
    _, logits = forward(m, x, ids)
    none = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    _, entropy, _, logprob, index = sam.token_logprobs(logits, none, top=top)
    return index[0].tolist(), logprob[0].tolist(), float(entropy[0])


def main():
    for objective in ("teacher", "tokens"):
        m, losses = train(objective=objective)
        print(f"{objective}: loss of a row {losses[0]:.4f} at the start, {losses[-1]:.4f} after {len(losses)} steps")
    x = torch.randn(1, m["W"].shape[0], device="cuda").to(m["W"].dtype)
    index, logprob, entropy = next_token(m, x, 0)
    print("next token:", ", ".join(f"{i} ({p:.2f})" for i, p in zip(index, logprob)), f"entropy {entropy:.2f}")


if __name__ == "__main__":
    main()
