"""Workspaces and limits of the token log probabilities, without a GPU."""
import ctypes

import pytest
import torch

import shape_adaptive_matrix_amd as sam
from tests.test_tokens_cpu import DEVICE, INVALID, MISALIGNED, WORKSPACE, L, P, fwd, grad


def test_short_workspace_is_refused():
    need = ctypes.c_uint64(0)
    assert L.sam_token_logprobs_workspace(sam.F32, 1, 131072, 20, ctypes.byref(need)) == 0 and need.value > 0
    big = dict(rows=1, V=131072, ldz=131072, top=20)
    assert fwd(**big, ws=None) == WORKSPACE and fwd(**big, n=need.value - 1) == WORKSPACE
    assert fwd(**big, ws=8 * P + 8) == MISALIGNED and fwd(**big, ws=P + 16) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks what is said without a GPU")
@pytest.mark.parametrize("V", [100, 16384, 16385, 131072])
def test_most_rows(V):
    """As many rows as the header says, and not one more."""
    rows, A = ((1 << 22) - 1) // ((V + 16383) // 16384), 1 << 44
    far = dict(V=V, ldz=V, z=A, tokens=2 * A, norm=5 * A, entropy=4 * A, top=0, best=None, index=None)
    assert fwd(rows=rows, logprob=3 * A, **far) == DEVICE and fwd(rows=rows + 1, logprob=3 * A, **far) == INVALID
    far.update(ldg=V, grad=11 * A, u=9 * A, v=10 * A)
    assert grad(rows=rows, **far) == DEVICE and grad(rows=rows + 1, **far) == INVALID
