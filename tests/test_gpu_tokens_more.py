"""Token log probabilities on the GPU: rows that few calls have, against their definition in 64 bits."""
import math

import pytest
import torch

import shape_adaptive_matrix_amd as sam
from tests import tokens_ref as ref
from tests.test_gpu_tokens import TYPES, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 3001, 70000])
@pytest.mark.parametrize("T", [1.0, 0.75, 1.9, 100.0])
def test_differences_past_the_range(T, V, dtype):
    """Logits at both ends of the type's range: their difference is none of FP32's numbers, its quotient by T may be."""
    R = 3
    z = torch.full((R, V), -3.0e38, device="cuda").to(TYPES[dtype])
    z[:, V // 2], z[1, 1], z[2, 5] = 3.0e38, -1.0e38, 0.0
    tokens = torch.tensor([0, 1, 5], dtype=torch.int32, device="cuda")
    logprob, entropy, norm, best, index = sam.token_logprobs(z, tokens, T, 8)
    order = ref.order(z)[:, :8]
    assert torch.equal(index, order.to(torch.int32))
    assert not entropy.any() and torch.equal(norm[:, 0], z[:, V // 2].float()) and not norm[:, 1].any()
    exact = (z.double() - z.double().amax(1, keepdim=True)) / T
    for got, want in ((logprob, exact.gather(1, tokens[:, None].long())[:, 0]), (best, exact.gather(1, order))):
        over = want.abs() >= torch.finfo(torch.float32).max * (1 + 2.0 ** -25)
        assert (got[over] == -math.inf).all() and got[~over].isfinite().all()
        # 1 / T as a float32, the halved difference and their product: half a step each.
        assert ((got[~over].double() - want[~over]).abs() <= 3 * 2.0 ** -24 * want[~over].abs()).all()
    one = torch.ones(R, device="cuda")
    grad = sam.token_logprobs_grad(z, tokens, norm, entropy, one, one, T)
    want = torch.zeros(R, V, device="cuda", dtype=torch.float64)
    want.scatter_(1, tokens[:, None].long(), 1.0 / float(torch.tensor(T, dtype=torch.float32)))
    want[:, V // 2] -= 1.0 / float(torch.tensor(T, dtype=torch.float32))
    assert torch.allclose(grad.double(), want, rtol=2 * ref.HALF_STEP[TYPES[dtype]], atol=0)
