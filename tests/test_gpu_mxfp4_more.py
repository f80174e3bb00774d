"""The 4-bit projection's less travelled ways on the GPU against its definition in 64 bits."""
import pytest
import torch

import shape_adaptive_matrix_amd as sam
from tests import mxfp4_ref as ref
from tests.test_gpu_mxfp4 import TYPES, normal, product_bound, weight

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


# Products whose K is cut: 4 ranges, 8, and fewer values than a range's; N of whole groups of four and not.
SPLIT = [(128, 4096, 4096), (65, 4096, 11008), (100, 1028, 4100), (96, 1030, 4096), (70, 333, 4000)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SPLIT, ids=str)
def test_linear_of_cut_products(shape, dtype):
    """Partial sums joined into results of either type, at every place and stride."""
    M, N, K = shape
    x = normal((M, K), dtype, 63)
    codes, scales, w = weight(N, K, 64)
    xq = ref.values(*ref.quantize(x), K)
    want, bound = xq @ w.t(), product_bound(xq, w)
    for out in {torch.float32, TYPES[dtype]}:
        need = sam._adapter_workspace_bytes("sam_linear_mxfp4_workspace", sam._value_code(x, "X"),
                                            sam._value_code(x.to(out), "Y"), M, N, K)
        assert need > 2 * 4 * M * N   # two or more partial sums of every result
        y = sam.linear_mxfp4(x, codes, scales, out_dtype=out)
        ref.close(y, want, bound)
        for pad, at in ((0, 1), (4, 0), (3, 2), (8, 4)):
            room = torch.full(((M + 1) * (N + pad) + 8,), -7.0, device="cuda", dtype=out)
            rows = room[at:at + (M + 1) * (N + pad)].view(M + 1, N + pad)
            sam.linear_mxfp4(x, codes, scales, Y=rows[:M, :N])
            assert torch.equal(rows[:M, :N], y)
            rows[:M, :N] = -7.0
            assert (room == -7).all()
