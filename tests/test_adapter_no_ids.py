"""The adapters' projection without adapters takes no ids."""
import pytest
import torch

import shape_adaptive_matrix_amd as sam
from tests.test_adapter_cpu import DEVICE, INVALID, backward, forward


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks what is said without a GPU")
def test_no_ids_reach_the_device_check():
    none = dict(n=0, A=None, B=None, scale=None, ids=None)
    assert forward(**none) == DEVICE and backward(**none, dA=None, dB=None) == DEVICE
    assert forward(ids=None) == INVALID and backward(ids=None) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (9, 520, 2048), (100, 300, 1000), (300, 512, 96), (700, 1000, 515)], ids=str)
def test_no_ids(M, N, K):
    """Through C with NULL: the bits that ids of any value give, forward and backward."""
    g = torch.Generator(device="cuda").manual_seed(3)
    K8 = (K + 7) // 8 * 8
    X, W, dY = (torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16) for s in ((M, K8), (K, N), (M, N)))
    A, B = (torch.zeros(0, 8, n, device="cuda", dtype=torch.bfloat16) for n in (K, N))
    ids = torch.randint(-5, 5, (M,), device="cuda", generator=g, dtype=torch.int32)
    want = sam.adapter_gemm(X[:, :K], W, A, B, ids)
    Y, dX = torch.empty(M, N, device="cuda"), torch.empty(M, K, device="cuda")
    ws = torch.empty(64 << 20, device="cuda", dtype=torch.uint8)
    L, s = sam.lib(), torch.cuda.current_stream().cuda_stream
    assert L.sam_adapter_gemm(sam.BF16, 0, M, N, K, 0, 8, X.data_ptr(), K8, W.data_ptr(), N, None, None, None, None, sam.F32,
                              Y.data_ptr(), N, ws.data_ptr(), ws.numel(), s) == 0, sam.last_error()
    assert L.sam_adapter_backward(sam.BF16, 0, M, N, K, 0, 8, dY.data_ptr(), N, X.data_ptr(), K8, W.data_ptr(), N, None, None,
                                  None, None, sam.F32, dX.data_ptr(), K, None, None, ws.data_ptr(), ws.numel(), s) == 0
    assert torch.equal(Y, want)
    wx = sam.adapter_backward(dY, X[:, :K], W, A, B, ids, need_dab=False)[0]
    assert torch.equal(dX, wx)
    exact = X[:, :K].double() @ W.double()
    bound = 2.0 ** -24 * (K + 64) * (X[:, :K].double().abs() @ W.double().abs())
    assert ((Y.double() - exact).abs() <= bound + 2.0 ** -24 * exact.abs()).all()
