"""The example that runs the 4-bit projection, the token log probabilities, the
distillation and the adapters together: every stage against 64 bits, from what
the stage was given."""
import importlib.util
import math
from pathlib import Path

import pytest
import torch

import shape_adaptive_matrix_amd as sam
from tests import distill_ref, mxfp4_ref, tokens_ref

pytestmark = pytest.mark.gpu

FILE = Path(__file__).resolve().parent.parent / "examples" / "recover_4bit.py"


def example():
    spec = importlib.util.spec_from_file_location("recover_4bit", FILE)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("objective", ["teacher", "tokens"])
@pytest.mark.parametrize("rows,hidden,vocabulary", [(40, 64, 500), (200, 96, 1003)])
def test_a_step(rows, hidden, vocabulary, objective):
    ex = example()
    m = ex.model(hidden=hidden, vocabulary=vocabulary, seed=3)
    m["B"] = torch.randn(m["B"].shape, device="cuda", generator=m["g"]) * 0.3
    X = torch.randn(rows, hidden, device="cuda", generator=m["g"]).bfloat16()
    ids = torch.randint(-1, 2, (rows,), device="cuda", generator=m["g"]).to(torch.int32)
    tokens = None
    if objective == "tokens":
        tokens = torch.randint(-1, vocabulary, (rows,), device="cuda", generator=m["g"]).to(torch.int32)
    s = ex.step(m, X, ids, top=20, tokens=tokens)

    code, scale = mxfp4_ref.quantize(m["head"].t())
    assert torch.equal(mxfp4_ref.unpack(m["codes"]), code) and torch.equal(m["scales"], scale)
    H = mxfp4_ref.values(code, scale, hidden)
    hq = mxfp4_ref.values(*mxfp4_ref.quantize(s["h"]), hidden)
    mxfp4_ref.close(s["logits"], hq @ H.t(), 2.0 ** -24 * (hidden + 32) * (hq.abs() @ H.abs().t()), "logits")

    weight = torch.full((rows,), 1.0 / rows, device="cuda")
    if objective == "teacher":
        loss, _, grad = distill_ref.reference(s["logits"], s["best"], s["index"], weight, 1.0)
        distill_ref.close(s["loss"], *loss, "loss")
        distill_ref.close(s["d_logits"], *grad, "d logits")
    else:
        want = tokens_ref.reference(s["logits"], tokens, 1.0, 0, -weight, -0.01 * weight)
        for name in ("logprob", "entropy", "norm"):
            tokens_ref.close(s[name], want[name], name)
        tokens_ref.close(s["d_logits"], want["grad"], "d logits")

    d = s["d_logits"].double()
    mxfp4_ref.close(s["d_h"], d @ H, 2.0 ** -24 * (vocabulary + 64) * (d.abs() @ H.abs()), "d h")

    # dA and dB: T is FP32 sums of exact products, then FP32 sums over rows.
    x, dh = X.double(), s["d_h"].double()
    u = 2.0 ** -24
    for a in range(2):
        r = ids == a
        Aa, Ba = m["A"][a].bfloat16().double(), m["B"][a].bfloat16().double()
        v, va = dh[r] @ Ba.t(), dh[r].abs() @ Ba.abs().t()
        t, ta = x[r] @ Aa.t(), x[r].abs() @ Aa.abs().t()
        n = int(r.sum()) + hidden + 64
        mxfp4_ref.close(s["dA"][a], v.t() @ x[r], 2 * u * n * (va.t() @ x[r].abs()), "dA")
        mxfp4_ref.close(s["dB"][a], t.t() @ dh[r], 2 * u * n * (ta.t() @ dh[r].abs()), "dB")


def test_it_runs_and_repeats():
    ex = example()
    for objective in ("teacher", "tokens"):
        m, losses = ex.train(steps=4, rows=64, objective=objective)
        assert all(math.isfinite(v) for v in losses)
        again = ex.train(steps=4, rows=64, objective=objective)
        assert again[1] == losses and torch.equal(again[0]["A"], m["A"]) and torch.equal(again[0]["B"], m["B"])   # the same bits
    x = torch.randn(1, 256, device="cuda").bfloat16()
    index, logprob, entropy = ex.next_token(m, x, 1)
    assert len(set(index)) == 5 and sorted(logprob, reverse=True) == logprob and 0 <= entropy <= math.log(2048) + 1e-5


def test_captured_step():
    """A whole step in a graph, replayed on other inputs."""
    ex = example()
    m = ex.model(seed=5)
    X = torch.randn(128, 256, device="cuda").bfloat16()
    ids = torch.zeros(128, dtype=torch.int32, device="cuda")
    tokens = torch.arange(128, device="cuda", dtype=torch.int32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ex.step(m, X, ids)
        ex.step(m, X, ids, tokens=tokens)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = ex.step(m, X, ids)
        b = ex.step(m, X, ids, tokens=tokens)
    for seed in (1, 2, 3):
        X.copy_(torch.randn(128, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)))
        want = ex.step(m, X, ids), ex.step(m, X, ids, tokens=tokens)
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((a, b), want):
            for k in w:
                assert torch.equal(got[k], w[k]), k
