"""What the distillation entry points refuse, without a GPU."""
import math

import pytest
import torch

import shape_adaptive_matrix_amd as sam

L = sam.lib()
P = 1 << 24   # made-up device addresses, refused before they are used
INVALID, MISALIGNED, DEVICE = -1, -2, -5


def loss(dtype=sam.F32, rows=4, V=100, top=5, z=P, ldz=100, td=sam.F32, t=2 * P, index=3 * P, weight=4 * P, T=1.0,
         loss=5 * P, lse=6 * P, **_):
    return L.sam_distill_loss(dtype, rows, V, top, z, ldz, td, t, index, weight, T, loss, lse, None)


def grad(dtype=sam.F32, rows=4, V=100, top=5, z=P, ldz=100, td=sam.F32, t=2 * P, index=3 * P, weight=4 * P, T=1.0,
         lse=6 * P, grad=7 * P, ldg=100, **_):
    return L.sam_distill_grad(dtype, rows, V, top, z, ldz, lse, td, t, index, weight, T, grad, ldg, None)


def both(dtype=sam.F32, rows=4, V=100, top=5, z=P, ldz=100, td=sam.F32, t=2 * P, index=3 * P, weight=4 * P, T=1.0,
         loss=5 * P, grad=7 * P, ldg=100, **_):
    return L.sam_distill(dtype, rows, V, top, z, ldz, td, t, index, weight, T, loss, grad, ldg, None)


REFUSED = [
    (dict(dtype=sam.MXFP8), INVALID), (dict(dtype=-1), INVALID), (dict(td=7), INVALID), (dict(rows=-1), INVALID),
    (dict(V=0), INVALID), (dict(V=1 << 31), INVALID), (dict(top=0), INVALID), (dict(top=1025), INVALID),
    (dict(ldz=99), INVALID), (dict(rows=1 << 31), INVALID), (dict(T=0.0), INVALID), (dict(T=-1.0), INVALID),
    (dict(T=2.0 ** -41), INVALID), (dict(T=2.0 ** 41), INVALID), (dict(T=math.nan), INVALID), (dict(T=math.inf), INVALID), (dict(z=None), INVALID), (dict(t=None), INVALID),
    (dict(index=None), INVALID), (dict(z=P + 2), MISALIGNED), (dict(t=2 * P + 2), MISALIGNED),
    (dict(index=3 * P + 2), MISALIGNED), (dict(weight=4 * P + 1), MISALIGNED),
]


@pytest.mark.parametrize("change,status", REFUSED, ids=[str(c) for c, _ in REFUSED])
def test_all_refuse(change, status):
    for call in (loss, grad, both):
        assert call(**change) == status, call.__name__
        assert sam.last_error()


def test_results_are_checked():
    assert loss(loss=None) == INVALID and loss(lse=None) == INVALID and both(loss=None) == INVALID
    assert grad(lse=None) == INVALID and grad(grad=None) == INVALID and both(grad=None) == INVALID
    assert loss(loss=6 * P) == INVALID and loss(lse=P) == INVALID and both(loss=3 * P) == INVALID
    for call in (grad, both):
        assert call(ldg=99) == INVALID
        assert call(grad=P + 400) == INVALID          # inside the logits, not in their place
        assert call(grad=P, ldg=101) == INVALID
        assert call(grad=3 * P) == INVALID and call(grad=4 * P) == INVALID
        assert call(grad=7 * P + 2) == MISALIGNED


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks what is said without a GPU")
def test_good_calls_reach_the_device_check():
    for call in (loss, grad, both):
        assert call() == DEVICE and call(weight=None) == DEVICE and call(dtype=sam.BF16, z=P + 2, td=sam.F16, t=2 * P + 2) == DEVICE
    assert grad(grad=P) == DEVICE and both(grad=P) == DEVICE


def test_no_rows():
    for call in (loss, grad, both):
        assert call(rows=0) == 0


@pytest.mark.parametrize("change", [
    dict(logits=torch.zeros(4, 50, dtype=torch.float64)), dict(logits=torch.zeros(50, 4).t()),
    dict(teacher=torch.zeros(3, 5)), dict(teacher=torch.zeros(4, 5, dtype=torch.int32)),
    dict(index=torch.zeros(4, 5, dtype=torch.int64)), dict(index=torch.zeros(4, 6, dtype=torch.int32)),
    dict(weight=torch.zeros(5)), dict(weight=torch.zeros(4, dtype=torch.float64)), dict()],
    ids=lambda c: ",".join(c) or "host tensors")
def test_binding_refuses(change):
    args = {**dict(logits=torch.zeros(4, 50), teacher=torch.zeros(4, 5), index=torch.zeros(4, 5, dtype=torch.int32),
                   weight=torch.ones(4)), **change}
    for call in (sam.distill_loss, sam.distill, lambda **a: sam.distill_grad(lse=torch.zeros(4), **a)):
        with pytest.raises((TypeError, ValueError)):
            call(**args)


@pytest.mark.parametrize("strides", [(0, 1), (1, 1), (49, 1)], ids=str)
def test_rows_that_share_memory_are_refused(strides, monkeypatch):
    """A row stride under a row's length was taken for a compact matrix."""
    shared = lambda: torch.zeros(4096).as_strided((4, 50), strides)  # noqa: E731
    rest = dict(teacher=torch.zeros(4, 5), index=torch.zeros(4, 5, dtype=torch.int32), weight=torch.ones(4))
    monkeypatch.setattr(sam, "_one_gpu", lambda *a: 0)   # host tensors, for results are looked at behind that check
    lse = torch.zeros(4)
    for call in (sam.distill_loss, sam.distill, lambda z, **a: sam.distill_grad(z, lse, **a)):
        with pytest.raises(ValueError, match="share memory"):
            call(shared(), **rest)
    for call in (sam.distill, lambda z, **a: sam.distill_grad(z, lse, **a)):
        with pytest.raises(ValueError, match="share memory"):
            call(torch.zeros(4, 50), **rest, grad=shared())


def test_gradient_needs_its_lse(monkeypatch):
    """None was replaced by new memory, and the gradient made of what it held."""
    monkeypatch.setattr(sam, "_one_gpu", lambda *a: 0)
    with pytest.raises(ValueError, match="lse"):
        sam.distill_grad(torch.zeros(4, 50), None, torch.zeros(4, 5), torch.zeros(4, 5, dtype=torch.int32))
