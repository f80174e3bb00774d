"""The example that runs the adapter projection and the distillation together."""
import importlib.util
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu

FILE = Path(__file__).resolve().parent.parent / "examples" / "distill_adapters.py"


def example():
    spec = importlib.util.spec_from_file_location("distill_adapters", FILE)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_distilled_adapters():
    ex = example()
    W, A, B, scale, losses = ex.train(steps=40)
    assert all(0 <= x < float("inf") for x in losses)
    assert losses[-1] < 0.5 * losses[0]
    again = ex.train(steps=40)[-1]
    assert again == losses                      # the same bits every time
    x = torch.randn(1, W.shape[0], device="cuda").to(W.dtype)
    plain = x.double() @ W.double()
    for user in (0, 2, -1):
        want = plain.clone()
        if user >= 0:
            want += (x.double() @ A[user].double().t()) @ B[user].double()
        got = ex.next_token_logits(x, W, A, B, scale, user)
        # FP32 sums over 256 values of size up to about 4, T in FP32.
        assert float((got.double() - want).abs().max()) < 2.0 ** -24 * 300 * 2 * float(
            x.double().abs() @ W.double().abs().max(1).values * (1 if user < 0 else 4))
