"""What the token log probabilities' entry points refuse, and their reference, without a GPU."""
import ctypes
import math

import pytest
import torch

import shape_adaptive_matrix_amd as sam
from tests import tokens_ref as ref

L = sam.lib()
P = 1 << 28   # made-up device addresses, refused before they are used
INVALID, MISALIGNED, WORKSPACE, DEVICE = -1, -2, -3, -5


def fwd(dtype=sam.F32, rows=4, V=100, top=5, z=P, ldz=100, tokens=2 * P, T=1.0, logprob=3 * P, entropy=4 * P, norm=5 * P,
        best=6 * P, index=7 * P, ws=8 * P, n=1 << 26, **_):
    return L.sam_token_logprobs(dtype, rows, V, top, z, ldz, tokens, T, logprob, entropy, norm, best, index, ws, n, None)


def grad(dtype=sam.F32, rows=4, V=100, z=P, ldz=100, tokens=2 * P, T=1.0, norm=5 * P, entropy=4 * P, u=9 * P, v=10 * P,
         grad=11 * P, ldg=100, **_):
    return L.sam_token_logprobs_grad(dtype, rows, V, z, ldz, tokens, T, norm, entropy, u, v, grad, ldg, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=sam.MXFP8), INVALID), (dict(dtype=-1), INVALID), (dict(rows=-1), INVALID), (dict(V=0), INVALID),
    (dict(V=1 << 31), INVALID), (dict(ldz=99), INVALID), (dict(rows=1 << 22), INVALID), (dict(T=0.0), INVALID),
    (dict(T=-1.0), INVALID), (dict(T=2.0 ** -41), INVALID), (dict(T=2.0 ** 41), INVALID), (dict(T=math.nan), INVALID),
    (dict(z=None), INVALID), (dict(tokens=None), INVALID), (dict(norm=None), INVALID), (dict(entropy=None), INVALID),
    (dict(z=P + 2), MISALIGNED), (dict(tokens=2 * P + 2), MISALIGNED), (dict(norm=5 * P + 1), MISALIGNED),
    (dict(entropy=4 * P + 2), MISALIGNED)], ids=str)
def test_both_refuse(change, status):
    for call in (fwd, grad):
        assert call(**change) == status, call.__name__
        assert sam.last_error()


@pytest.mark.parametrize("change,status", [
    (dict(top=-1), INVALID), (dict(top=129, V=1000, ldz=1000), INVALID), (dict(top=101), INVALID), (dict(logprob=None), INVALID),
    (dict(best=None), INVALID), (dict(index=None), INVALID), (dict(logprob=P), INVALID), (dict(entropy=3 * P + 4), INVALID),
    (dict(index=6 * P + 16), INVALID), (dict(norm=2 * P), INVALID)], ids=str)
def test_forward_refuses(change, status):
    assert fwd(**change) == status


def test_workspace():
    need = ctypes.c_uint64(7)
    assert L.sam_token_logprobs_workspace(sam.F32, 1, 131072, 20, None) == INVALID
    assert L.sam_token_logprobs_workspace(sam.F32, 1, 131072, 129, ctypes.byref(need)) == INVALID
    assert L.sam_token_logprobs_workspace(sam.F32, 1, 131072, 20, ctypes.byref(need)) == 0
    if need.value:
        big = dict(rows=1, V=131072, ldz=131072, top=20)
        assert fwd(**big, ws=None) == WORKSPACE and fwd(**big, n=need.value - 1) == WORKSPACE
        assert fwd(**big, ws=8 * P + 8) == MISALIGNED and fwd(**big, ws=P + 16) == INVALID


def test_gradient_refuses():
    assert grad(grad=None) == INVALID and grad(ldg=99) == INVALID and grad(grad=11 * P + 2) == MISALIGNED
    assert grad(grad=P + 400) == INVALID and grad(grad=P, ldg=101) == INVALID   # inside the logits, not in their place
    assert grad(grad=5 * P) == INVALID and grad(grad=9 * P) == INVALID and grad(grad=10 * P) == INVALID
    assert grad(u=9 * P + 1) == MISALIGNED


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks what is said without a GPU")
def test_good_calls_reach_the_device_check():
    assert fwd() == DEVICE and fwd(top=0, best=None, index=None) == DEVICE and fwd(dtype=sam.BF16, z=P + 2) == DEVICE
    assert fwd(rows=1, ldz=0) == DEVICE
    assert grad() == DEVICE and grad(grad=P) == DEVICE and grad(u=None) == DEVICE
    assert grad(v=None, entropy=None) == DEVICE and grad(rows=1, ldz=0, ldg=0, grad=P) == DEVICE


def test_no_rows():
    assert fwd(rows=0) == 0 and grad(rows=0) == 0


@pytest.mark.parametrize("change", [
    dict(logits=torch.zeros(4, 50).double()), dict(logits=torch.zeros(50, 4).t()), dict(tokens=torch.zeros(4)),
    dict(tokens=torch.zeros(5, dtype=torch.int32)), dict(tokens=torch.zeros(4, dtype=torch.int64)),
    dict(tokens=torch.zeros(8, dtype=torch.int32)[::2]), dict(logits=torch.zeros(1, 50).expand(4, 50)), dict()],
    ids=lambda c: ",".join(c) or "host")
def test_binding_refuses(change):
    t = {**dict(logits=torch.zeros(4, 50), tokens=torch.zeros(4, dtype=torch.int32)), **change}
    for call in (lambda: sam.token_logprobs(t["logits"], t["tokens"], top=3),
                 lambda: sam.token_logprobs_grad(t["logits"], t["tokens"], torch.zeros(4, 2), torch.zeros(4), torch.zeros(4))):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_gradient_needs_what_the_forward_pass_gave(monkeypatch):
    monkeypatch.setattr(sam, "_one_gpu", lambda *a: 0)   # host tensors, for these are looked at behind that check
    monkeypatch.setattr(sam, "_elsewhere", lambda d: None)
    z, t = torch.zeros(4, 50), torch.zeros(4, dtype=torch.int32)
    for more in (dict(norm=None), dict(norm=torch.zeros(4, 2), dentropy=torch.zeros(4)), dict(norm=torch.zeros(4)),
                 dict(norm=torch.zeros(4, 2), dlogprob=torch.zeros(3)), dict(norm=torch.zeros(4, 2).double())):
        with pytest.raises(ValueError):
            sam.token_logprobs_grad(z, t, **more)


def test_reference():
    """By hand: probabilities 1/2, 1/4, 1/4, 0; and the gradient against differences in 64 bits."""
    z = torch.tensor([[math.log(2.0), 0.0, -math.inf, 0.0]], dtype=torch.float64)
    r = ref.reference(z, torch.tensor([1]), 1.0, top=4)
    assert abs(float(r["logprob"][0]) + math.log(4)) < 1e-15 and abs(float(r["entropy"][0]) - 1.5 * math.log(2)) < 1e-15
    assert r["top_index"].tolist() == [[0, 1, 3, 2]]
    torch.manual_seed(1)
    z, t = torch.randn(3, 7, dtype=torch.float64), torch.tensor([2, 6, -1])
    u, v = torch.randn(3), torch.randn(3)
    got = ref.reference(z, t, 0.75, u=u, v=v)["grad"][0]
    h = 1e-6
    for j in range(7):
        step = torch.zeros_like(z)
        step[:, j] = h
        a, b = (ref.reference(z + s, t, 0.75) for s in (step, -step))
        diff = sum(w.double() * (a[k][0] - b[k][0]) / (2 * h) for w, k in ((u, "logprob"), (v, "entropy")))
        assert torch.allclose(diff, got[:, j], atol=1e-8)
