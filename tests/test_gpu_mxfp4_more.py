"""The 4-bit projection's less travelled ways on the GPU against its definition in 64 bits."""
import pytest
import torch

import shape_adaptive_matrix_amd as sam
from tests import mxfp4_ref as ref
from tests.test_gpu_mxfp4 import TYPES, normal, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad", [1, 2, 5, 8])
@pytest.mark.parametrize("M,N,K", [(2048, 75, 3243), (300, 77, 131), (1000, 1866, 515)], ids=str)
def test_backward_into_padded_rows(M, N, K, pad, dtype):
    """K of three values past whole 16-byte pieces, results of every stride."""
    codes, scales, w = weight(N, K, 61)
    dy = normal((M, N), dtype, 62)
    want = dy.double() @ w
    bound = 2.0 ** -24 * (N + 64) * (dy.double().abs() @ w.abs())
    dx = torch.full((M + 1, K + pad), -7.0, device="cuda").to(TYPES[dtype])
    sam.linear_mxfp4_backward(dy, codes, scales, dX=dx[:M, :K])
    ref.close(dx[:M, :K], want, bound)
    assert (dx[M] == -7).all() and (dx[:, K:] == -7).all()
