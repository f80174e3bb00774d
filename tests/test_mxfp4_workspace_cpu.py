"""What the 4-bit projection's backward pass asks for as workspace holds what its products take, without a GPU."""
import ctypes

import pytest

import shape_adaptive_matrix_amd as sam

L = sam.lib()
LARGEST = 0x7FFFFFF0 // (257 * 4)


def size(call, *args):
    n = ctypes.c_uint64()
    assert call(*args, ctypes.byref(n)) == 0, sam.last_error()
    return n.value


def up(n, to):
    return (n + to - 1) // to * to


def needed(dtype, M, N, K, lddy, lddx):
    """The read-back weight beside what the product of these strides takes."""
    f32 = dtype == sam.F32
    row = up(K, 4 if f32 else 8)
    weight = up(N * row * (4 if f32 else 2), 256)
    if f32:
        return weight + size(L.sam_gemm_ex_workspace, dtype, 0, 0, M, K, N, lddy, row, lddx, 1.0, 0.0)
    return weight + size(L.sam_adapter_gemm_workspace, dtype, 0, M, K, N, 0, 1, lddy, row)


# Every residue of N and K to a 16-byte piece, with sizes of few, some and many tiles.
@pytest.mark.parametrize("dtype", [sam.F32, sam.BF16, sam.F16])
@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (33, 320, 512), (600, 1856, 2280), (2048, 72, 3240), (4096, 4096, 11000)], ids=str)
def test_query_holds_every_stride(M, N, K, dtype):
    for n in range(N, N + 8):
        for k in range(K, K + 8):
            query = size(L.sam_linear_mxfp4_backward_workspace, dtype, sam.F32, M, n, k)
            for lddy in (n, n + 1, n + 2, n + 5, up(n + 1, 8)):
                for lddx in (k, k + 1, k + 2, k + 5, up(k + 1, 8)):
                    assert query >= needed(dtype, M, n, k, lddy, lddx), (n, k, lddy, lddx)


@pytest.mark.parametrize("dtype", [sam.F32, sam.BF16, sam.F16])
def test_largest_sizes(dtype):
    assert size(L.sam_linear_mxfp4_backward_workspace, dtype, sam.F32, 2, LARGEST, 64) > 0
    assert size(L.sam_linear_mxfp4_backward_workspace, dtype, sam.F32, 2, 64, LARGEST // 8 * 8) > 0


@pytest.mark.parametrize("dtype", [sam.F32, sam.BF16, sam.F16])
@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (33, 320, 512), (600, 1856, 2280), (2048, 72, 3240)], ids=str)
def test_query_of_given_strides(M, N, K, dtype):
    """No more than these strides need, and never more than for any stride."""
    for n in (N, N + 1, N + 3, N + 7):
        for k in (K, K + 1, K + 3, K + 7):
            query = size(L.sam_linear_mxfp4_backward_workspace, dtype, sam.F32, M, n, k)
            for lddy in (n, n + 1, n + 2, n + 5, up(n + 1, 8)):
                for lddx in (k, k + 1, k + 2, k + 5, up(k + 1, 8)):
                    need = needed(dtype, M, n, k, *((n, k) if M == 1 else (lddy, lddx)))
                    got = size(L.sam_linear_mxfp4_backward_workspace_strided, dtype, sam.F32, M, n, k, lddy, lddx)
                    assert need <= got <= min(query, up(need, 256)), (n, k, lddy, lddx)


def test_compact_gradient_is_not_copied():
    """A training batch's gradient of a large vocabulary: the weight and little else."""
    M, N, K = 4096, 131072, 4096
    assert size(L.sam_linear_mxfp4_backward_workspace_strided, sam.BF16, sam.BF16, M, N, K, N, K) < 1.01 * 2 * N * K


def test_strided_query_refuses():
    n = ctypes.c_uint64(7)
    q = L.sam_linear_mxfp4_backward_workspace_strided
    assert q(sam.BF16, sam.F32, 4, 60, 100, 60, 100, None) == -1
    for lddy, lddx in ((59, 100), (60, 99), (LARGEST + 1, 100), (60, LARGEST + 1)):
        assert q(sam.BF16, sam.F32, 4, 60, 100, lddy, lddx, ctypes.byref(n)) == -1
    assert q(sam.BF16, sam.F32, 0, 60, 100, 60, 100, ctypes.byref(n)) == 0 and n.value == 0
    assert q(sam.BF16, sam.F32, 1, 60, 100, 0, 0, ctypes.byref(n)) == 0 and n.value > 0
