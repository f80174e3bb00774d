"""What the adapter entry points refuse, and their workspace queries, without a
GPU: everything is rejected on the host before any device call."""
import ctypes
import subprocess
import sys
from pathlib import Path

import pytest
import torch

import shape_adaptive_matrix_amd as sam

L = sam.lib()
P = 1 << 20   # made-up device addresses, 16-byte aligned and far apart: refused before they are used


def forward(dtype=sam.BF16, trans=0, M=8, N=64, K=64, n=2, r=8, X=P, ldx=64, W=2 * P, ldw=64, A=3 * P, B=4 * P,
            ids=5 * P, scale=6 * P, out=sam.F32, Y=7 * P, ldy=64, ws=8 * P, wsb=1 << 19):
    return L.sam_adapter_gemm(dtype, trans, M, N, K, n, r, X, ldx, W, ldw, A, B, ids, scale, out, Y, ldy, ws, wsb, None)


def backward(dtype=sam.BF16, trans=0, M=8, N=64, K=64, n=2, r=8, dY=P, lddy=64, X=2 * P, ldx=64, W=3 * P, ldw=64,
             A=4 * P, B=5 * P, ids=6 * P, scale=None, out=sam.F32, dX=7 * P, lddx=64, dA=8 * P, dB=9 * P, ws=10 * P,
             wsb=1 << 19):
    return L.sam_adapter_backward(dtype, trans, M, N, K, n, r, dY, lddy, X, ldx, W, ldw, A, B, ids, scale, out, dX, lddx,
                                  dA, dB, ws, wsb, None)


INVALID, MISALIGNED, WORKSPACE, DEVICE = -1, -2, -3, -5

REFUSED = [
    (dict(dtype=sam.F32), INVALID), (dict(dtype=sam.MXFP8), INVALID), (dict(trans=2), INVALID),
    (dict(out=sam.F16), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(n=-1), INVALID),
    (dict(r=0), INVALID), (dict(r=129), INVALID), (dict(ldx=63), INVALID), (dict(ldw=63), INVALID),
    (dict(M=1 << 31), INVALID), (dict(ldx=1 << 23), INVALID), (dict(X=None), INVALID), (dict(W=None), INVALID),
    (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(ids=None), INVALID), (dict(X=P + 8), MISALIGNED),
    (dict(W=2 * P + 2), MISALIGNED), (dict(ids=5 * P + 2), MISALIGNED), (dict(wsb=16), WORKSPACE),
    (dict(ws=None), WORKSPACE),
]


@pytest.mark.parametrize("change,status", REFUSED, ids=[str(c) for c, _ in REFUSED])
def test_both_passes_refuse(change, status):
    for call in (forward, backward):
        assert call(**change) == status, call.__name__
        assert sam.last_error()


def test_forward_refuses():
    for change, status in [(dict(ldy=63), INVALID), (dict(Y=None), INVALID), (dict(Y=P), INVALID), (dict(Y=8 * P), INVALID),
                           (dict(Y=5 * P), INVALID), (dict(Y=7 * P + 4), MISALIGNED), (dict(scale=6 * P + 1), MISALIGNED),
                           (dict(ws=4 * P), INVALID)]:
        assert forward(**change) == status, change


def test_backward_refuses():
    for change, status in [(dict(lddy=63), INVALID), (dict(lddx=63), INVALID), (dict(dA=None), INVALID),
                           (dict(dB=None), INVALID), (dict(dA=9 * P), INVALID), (dict(dX=2 * P), INVALID),
                           (dict(dB=10 * P), INVALID), (dict(dA=8 * P + 4), MISALIGNED)]:
        assert backward(**change) == status, change


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks what is said without a GPU")
def test_good_calls_reach_the_device_check():
    assert forward() == DEVICE and backward() == DEVICE
    assert backward(dX=None) == DEVICE and backward(dA=None, dB=None) == DEVICE
    assert forward(n=0, A=None, B=None, scale=None) == DEVICE


def test_nothing_to_do():
    assert forward(M=0) == 0
    assert backward(dX=None, dA=None, dB=None) == 0


def test_workspace_queries():
    b = ctypes.c_uint64()
    q = lambda *a: L.sam_adapter_gemm_workspace(*a, ctypes.byref(b))  # noqa: E731
    assert q(sam.BF16, 0, 4096, 4096, 4096, 8, 16, 4096, 4096) == 0
    # T's partial sums (FP32) and what its rounded form takes, not a copy of any operand.
    assert 4096 * 16 * 4 <= b.value < 4096 * 4096 * 2
    assert q(sam.BF16, 0, 0, 64, 64, 8, 16, 64, 64) == 0 and b.value == 0
    assert q(sam.F32, 0, 8, 64, 64, 8, 16, 64, 64) == INVALID
    assert L.sam_adapter_gemm_workspace(sam.BF16, 0, 8, 64, 64, 8, 16, 64, 64, None) == INVALID
    q = lambda *a: L.sam_adapter_backward_workspace(*a, ctypes.byref(b))  # noqa: E731
    assert q(sam.BF16, 0, 64, 64, 64, 2, 8, 64, 64, 64, 1, 1) == 0
    whole = b.value
    assert q(sam.BF16, 0, 64, 64, 64, 2, 8, 64, 64, 64, 0, 1) == 0 and b.value <= whole


def test_w_with_padded_rows_takes_no_copy():
    """Rows along the product's columns: read in place; along its K: copied."""
    def need(trans_w, M, N, K, ldw, back):
        b = ctypes.c_uint64()
        if back:
            assert L.sam_adapter_backward_workspace(sam.BF16, trans_w, M, N, K, 2, 16, N, K, ldw, 1, 0, ctypes.byref(b)) == 0
        else:
            assert L.sam_adapter_gemm_workspace(sam.BF16, trans_w, M, N, K, 2, 16, K, ldw, ctypes.byref(b)) == 0
        return b.value

    copy = 2 * 512 * 4008
    assert need(0, 40, 4001, 512, 4001, 0) - need(0, 40, 4001, 512, 4008, 0) >= copy
    assert need(1, 40, 512, 4001, 4001, 0) == need(1, 40, 512, 4001, 4008, 0)
    assert need(1, 40, 512, 4001, 4001, 1) - need(1, 40, 512, 4001, 4008, 1) >= copy
    assert need(0, 40, 4001, 512, 4001, 1) == need(0, 40, 4001, 512, 4008, 1)


def _tensors():
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    return dict(X=t(4, 32), W=t(32, 48), A=t(2, 8, 32), B=t(2, 8, 48), ids=torch.zeros(4, dtype=torch.int32),
                scale=torch.ones(2))


@pytest.mark.parametrize("change", [
    dict(X=torch.zeros(4, 32)), dict(W=torch.zeros(32, 48, dtype=torch.float16)), dict(W=torch.zeros(48, 32, dtype=torch.bfloat16)),
    dict(A=torch.zeros(2, 4, 32, dtype=torch.bfloat16)), dict(B=torch.zeros(2, 48, 8, dtype=torch.bfloat16).transpose(1, 2)),
    dict(ids=torch.zeros(4, dtype=torch.int64)), dict(ids=torch.zeros(3, dtype=torch.int32)), dict(scale=torch.ones(3)),
    dict(scale=torch.ones(2, dtype=torch.bfloat16)), dict(out_dtype=torch.float16),
    dict(X=torch.zeros(32, 4, dtype=torch.bfloat16).t()), dict()], ids=lambda c: ",".join(c) or "host tensors")
def test_binding_refuses(change):
    args = {**_tensors(), **change}
    with pytest.raises((TypeError, ValueError)):
        sam.adapter_gemm(**args)
    dY = torch.zeros(4, 48, dtype=torch.bfloat16)
    with pytest.raises((TypeError, ValueError)):
        sam.adapter_backward(dY, **args)


@pytest.mark.parametrize("N,K", [(72, 64), (512, 64), (64, 512), (4096, 4096), (2049, 1025)])
def test_no_rows_is_answered(N, K):
    """In a process of its own: the library must not end it."""
    code = f"""
import ctypes, shape_adaptive_matrix_amd as sam
L, b, P = sam.lib(), ctypes.c_uint64(), 1 << 20
for trans in (0, 1):
    ldw = {K} if trans else {N}
    for n in (0, 1, 3):
        assert L.sam_adapter_gemm_workspace(sam.BF16, trans, 0, {N}, {K}, n, 8, {K}, ldw, ctypes.byref(b)) == 0
        for dx, dab in ((0, 0), (0, 1), (1, 0), (1, 1)):
            assert L.sam_adapter_backward_workspace(sam.F16, trans, 0, {N}, {K}, n, 8, {N}, {K}, ldw, dx, dab,
                                                    ctypes.byref(b)) == 0
            if dab and n:
                assert 0 < b.value < 1 << 30
    # Refused for its short workspace, so the layout is made and nothing is launched.
    assert L.sam_adapter_backward(sam.BF16, trans, 0, {N}, {K}, 3, 8, P, {N}, 2 * P, {K}, None, ldw, 4 * P, 5 * P, 6 * P,
                                  None, sam.F32, None, {K}, 8 * P, 12 * P, 16 * P, 1, None) == -3
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parent.parent, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-500:]


SHARED = [(0, 1), (1, 1), (31, 1)]   # strides of rows of 32 and 48 that share memory: broadcast, and overlapping windows


@pytest.mark.parametrize("strides", SHARED, ids=str)
def test_rows_that_share_memory_are_refused(strides, monkeypatch):
    """A row stride under a row's length was taken for a compact matrix."""
    shared = lambda rows, cols, like: like.new_zeros(4096).as_strided((rows, cols), strides)  # noqa: E731
    args = _tensors()
    h, f = args["X"], args["scale"]
    dY = h.new_zeros(4, 48)
    monkeypatch.setattr(sam, "_one_gpu", lambda *a: 0)   # host tensors, for results are looked at behind that check
    for change in (dict(X=shared(4, 32, h)), dict(W=shared(32, 48, h)), dict(W=shared(48, 32, h), trans_w=True)):
        with pytest.raises(ValueError, match="share memory"):
            sam.adapter_gemm(**{**args, **change})
        with pytest.raises(ValueError, match="share memory"):
            sam.adapter_backward(dY, **{**args, **change})
    with pytest.raises(ValueError, match="share memory"):
        sam.adapter_gemm(**args, Y=shared(4, 48, f))
    with pytest.raises(ValueError, match="share memory"):
        sam.adapter_backward(shared(4, 48, h), **args)
    with pytest.raises(ValueError, match="share memory"):
        sam.adapter_backward(dY, **args, dX=shared(4, 32, f))
    # One row, one column, or none shares nothing.
    for rows, cols, st in ((1, 32, (0, 1)), (1, 32, (7, 1)), (4, 1, (1, 0)), (0, 32, (0, 1)), (4, 32, (32, 1)), (4, 32, (40, 1))):
        assert sam._matrix(h.new_zeros(4096).as_strided((rows, cols), st), "X")[:2] == (rows, cols)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks what is said without a GPU")
def test_a_single_row_has_any_stride():
    """The last position of one long sequence: its stride is the sequence's length times K."""
    far = 300 * 8192
    assert forward(M=1, ldx=far) == DEVICE and forward(M=1, ldy=far) == DEVICE
    assert backward(M=1, ldx=far) == DEVICE and backward(M=1, lddy=far) == DEVICE and backward(M=1, lddx=far) == DEVICE
    assert forward(K=1, ldw=far) == DEVICE and forward(trans=1, N=1, ldw=far) == DEVICE
    assert forward(M=2, ldx=far) == INVALID and forward(K=2, ldw=far) == INVALID and backward(M=2, lddy=far) == INVALID
    assert forward(M=1, ldx=63) == INVALID and backward(M=1, lddy=63) == INVALID
    b = [ctypes.c_uint64() for _ in range(3)]
    for q, ld in zip(b, (64, 67, far)):   # no copy of it either
        assert L.sam_adapter_gemm_workspace(sam.BF16, 0, 1, 64, 64, 2, 8, ld, 64, ctypes.byref(q)) == 0
    assert b[0].value == b[1].value == b[2].value


@pytest.mark.parametrize("M,n,parts", [(64, 1000, 0), (128, 4, 0), (1025, 1000, 31), (1025, 3, 19), (5000, 50000, 154)])
def test_partials_for_adapters_that_have_them(M, n, parts):
    """dA and dB of an adapter with no more rows than a chunk (64, or all of up
    to 128) are written at once: partials do not grow with the adapters."""
    K, N, r = 1024, 1024, 16
    b = ctypes.c_uint64()
    assert L.sam_adapter_backward_workspace(sam.BF16, 0, M, N, K, n, r, N, K, N, 0, 1, ctypes.byref(b)) == 0
    rest = 2 * 4 * M * r * 32 + 3 * 2 * M * r + 4 * (4 * n + 8 * M) + 16 * (M // 64 + n) + (1 << 16)   # T's sums, lists
    assert b.value <= parts * 4 * r * (K + N) + rest
