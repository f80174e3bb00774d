"""What the MXFP4 entry points refuse, and their reference, without a GPU."""
import ctypes

import pytest
import torch

import shape_adaptive_matrix_amd as sam
from tests import mxfp4_ref as ref

L = sam.lib()
P = 1 << 24   # made-up device addresses, refused before they are used
INVALID, MISALIGNED, WORKSPACE, DEVICE = -1, -2, -3, -5


def quant(dtype=sam.BF16, trans=0, rows=4, K=100, X=P, ldx=100, codes=2 * P, scales=3 * P):
    return L.sam_quantize_mxfp4(dtype, trans, rows, K, X, ldx, codes, scales, None)


def dequant(dtype=sam.BF16, rows=4, K=100, X=P, ldx=100, codes=2 * P, scales=3 * P):
    return L.sam_dequantize_mxfp4(dtype, rows, K, codes, scales, X, ldx, None)


def linear(dtype=sam.BF16, M=100, N=60, K=100, X=P, ldx=100, codes=2 * P, scales=3 * P, out=sam.F32, Y=4 * P, ldy=60,
           ws=5 * P, n=1 << 23):
    return L.sam_linear_mxfp4(dtype, M, N, K, X, ldx, codes, scales, out, Y, ldy, ws, n, None)


def back(dtype=sam.BF16, M=100, N=60, K=100, X=P, ldx=60, codes=2 * P, scales=3 * P, out=sam.F32, Y=4 * P, ldy=100,
         ws=5 * P, n=1 << 23):
    return L.sam_linear_mxfp4_backward(dtype, M, N, K, X, ldx, codes, scales, out, Y, ldy, ws, n, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=sam.MXFP4), INVALID), (dict(dtype=-1), INVALID), (dict(rows=-1), INVALID), (dict(K=0), INVALID),
    (dict(K=1 << 31), INVALID), (dict(rows=1 << 30, K=65), INVALID), (dict(rows=(1 << 30) - 1, K=64, ldx=64), INVALID), (dict(ldx=99), INVALID), (dict(X=None), INVALID),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(X=P + 1), MISALIGNED),
    (dict(dtype=sam.F32, X=P + 2), MISALIGNED), (dict(codes=2 * P + 8), MISALIGNED)], ids=str)
def test_tensors_refuse(change, status):
    for call in (quant, dequant):
        assert call(**change) == status, call.__name__
        assert sam.last_error()


def test_tensors_more():
    assert quant(trans=2) == INVALID
    assert quant(trans=1, ldx=3) == INVALID
    assert quant(codes=P + 16) == INVALID and quant(scales=P + 1) == INVALID and quant(scales=2 * P + 3) == INVALID
    assert dequant(X=2 * P + 16) == INVALID and dequant(X=3 * P) == INVALID
    assert quant(rows=0) == 0 and dequant(rows=0) == 0


@pytest.mark.parametrize("change,status", [
    (dict(dtype=sam.MXFP8), INVALID), (dict(out=sam.F16), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID),
    (dict(K=0), INVALID), (dict(N=3 << 20), INVALID), (dict(K=3 << 20), INVALID), (dict(M=1 << 31), INVALID),
    (dict(M=1 << 30, K=128), INVALID), (dict(M=1 << 29, N=32, K=32), INVALID), (dict(N=1 << 20, K=1 << 16), INVALID),
    (dict(ldx=59), INVALID), (dict(ldy=59), INVALID), (dict(X=None), INVALID),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(Y=None), INVALID), (dict(X=P + 1), MISALIGNED),
    (dict(codes=2 * P + 4), MISALIGNED), (dict(Y=4 * P + 2), MISALIGNED), (dict(ws=5 * P + 8), MISALIGNED),
    (dict(Y=P), INVALID), (dict(Y=2 * P), INVALID), (dict(Y=3 * P + 16), INVALID), (dict(ws=4 * P + 256), INVALID),
    (dict(ws=P + 16), INVALID), (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE)], ids=str)
def test_products_refuse(change, status):
    for call in (linear, back):
        assert call(**change) == status, call.__name__
        assert sam.last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks what is said without a GPU")
def test_good_calls_reach_the_device_check():
    assert quant() == DEVICE and quant(trans=1, ldx=4) == DEVICE and quant(X=P + 2) == DEVICE and dequant() == DEVICE
    assert quant(rows=1, ldx=0) == DEVICE and dequant(rows=1, ldx=0) == DEVICE
    for call in (linear, back):
        assert call() == DEVICE and call(out=sam.BF16) == DEVICE and call(dtype=sam.F32) == DEVICE
        assert call(M=1, ldx=0, ldy=1 << 50) == DEVICE and call(scales=3 * P + 1) == DEVICE
    assert linear(X=P + 2, Y=4 * P + 4) == DEVICE


def test_no_rows_and_workspaces():
    n = ctypes.c_uint64(7)
    for call, ws in ((linear, L.sam_linear_mxfp4_workspace), (back, L.sam_linear_mxfp4_backward_workspace)):
        assert call(M=0) == 0 and call(M=0, ws=None) == 0
        assert ws(sam.BF16, sam.F32, 0, 60, 100, ctypes.byref(n)) == 0 and n.value == 0
        assert ws(sam.BF16, sam.F32, 4, 60, 100, None) == INVALID
        assert ws(sam.BF16, sam.F16, 4, 60, 100, ctypes.byref(n)) == INVALID
        assert ws(sam.BF16, sam.F32, 4, 0, 100, ctypes.byref(n)) == INVALID


u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731


@pytest.mark.parametrize("change", [
    dict(codes=u8(8, 30)), dict(codes=u8(8, 32).t()), dict(codes=u8(8, 64)[:, :32]), dict(codes=u8(8, 32).to(torch.int8)),
    dict(scales=u8(8, 3)), dict(scales=u8(7, 2)), dict(scales=torch.zeros(8, 2)), dict()], ids=lambda c: ",".join(c) or "host")
def test_binding_refuses(change):
    t = {**dict(codes=u8(8, 32), scales=u8(8, 2)), **change}
    for call in (lambda: sam.dequantize_mxfp4(t["codes"], t["scales"]), lambda: sam.quantize_mxfp4(torch.zeros(8, 50), **t),
                 lambda: sam.linear_mxfp4(torch.zeros(3, 50), t["codes"], t["scales"]),
                 lambda: sam.linear_mxfp4_backward(torch.zeros(3, 8), t["codes"], t["scales"], 50)):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_binding_refuses_shapes():
    c, s = u8(8, 32), u8(8, 2)
    for call in (lambda: sam.dequantize_mxfp4(c, s, 32), lambda: sam.dequantize_mxfp4(c, s, 65),
                 lambda: sam.linear_mxfp4(torch.zeros(3, 65), c, s), lambda: sam.linear_mxfp4(torch.zeros(3, 50).double(), c, s),
                 lambda: sam.linear_mxfp4_backward(torch.zeros(3, 9), c, s, 50),
                 lambda: sam.quantize_mxfp4(torch.zeros(8, 50, 2)), lambda: sam.quantize_mxfp4(torch.zeros(100, 8)[:, ::2])):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_reference():
    """By hand: a block whose largest value is 7 (s = 0), every border between codes, and its neighbours."""
    x = torch.zeros(1, 40)
    x[0, :16] = torch.tensor([7.0, 0.25, 0.26, 0.75, 0.74, 1.25, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, -0.25, -5.5, -0.0, 1.0])
    x[0, 32:34] = torch.tensor([-2.0 ** -130, 2.0 ** -127])
    code, scale = ref.quantize(x)
    assert scale.tolist() == [[127, 0]]
    assert code[0, :16].tolist() == [7, 0, 1, 2, 1, 2, 4, 4, 5, 6, 6, 7, 8, 15, 8, 2]
    assert code[0, 32:34].tolist() == [8, 2]
    assert ref.values(code, scale, 40)[0, [0, 3, 13, 33]].tolist() == [6.0, 1.0, -6.0, 2.0 ** -127]
    assert torch.equal(ref.unpack(ref.pack(code)), code)
