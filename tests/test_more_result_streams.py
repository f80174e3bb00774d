"""The checks of test_result_streams for the 4-bit projection and the token log probabilities."""
import pytest
import torch

import shape_adaptive_matrix_amd as sam
from tests import test_result_streams as base

M, K, N = 1024, 512, 2048


def calls(device):
    X = torch.zeros(M, K, dtype=torch.bfloat16, device=device)
    dY = torch.zeros(M, N, dtype=torch.bfloat16, device=device)
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device=device)
    scales = torch.zeros(N, K // 32, dtype=torch.uint8, device=device)
    tokens = torch.zeros(M, dtype=torch.int32, device=device)
    few = torch.zeros(4, 200000, device=device)   # rows cut over workgroups: a workspace
    norm, one = torch.zeros(M, 2, device=device), torch.ones(M, device=device)
    return [
        ("quantize", lambda s: sam.quantize_mxfp4(X, stream=s)),
        ("dequantize", lambda s: sam.dequantize_mxfp4(codes, scales, stream=s)),
        ("linear", lambda s: sam.linear_mxfp4(X, codes, scales, stream=s)),
        ("linear of bf16", lambda s: sam.linear_mxfp4(X, codes, scales, out_dtype=X.dtype, stream=s)),
        ("linear of few rows", lambda s: sam.linear_mxfp4(X[:16], codes, scales, stream=s)),
        ("linear backward", lambda s: sam.linear_mxfp4_backward(dY, codes, scales, stream=s)),
        ("token_logprobs", lambda s: sam.token_logprobs(dY, tokens, stream=s)),
        ("token_logprobs with alternatives", lambda s: sam.token_logprobs(dY, tokens, top=5, stream=s)),
        ("token_logprobs of few rows", lambda s: sam.token_logprobs(few, tokens[:4], top=5, stream=s)),
        ("token_logprobs_grad", lambda s: sam.token_logprobs_grad(dY, tokens, norm, None, one, stream=s)),
    ]


NAMES = [n for n, _ in calls("cpu")]


@pytest.mark.skipif(torch.cuda.is_available(), reason="host tensors: checks what is done without a GPU")
@pytest.mark.parametrize("name", NAMES)
def test_results_are_allocated_on_the_stream(name, monkeypatch):
    monkeypatch.setattr(base, "calls", calls)
    monkeypatch.setattr(sam, "_elsewhere", lambda d: None)
    base.test_results_are_allocated_on_the_stream(name, monkeypatch)


# Of few rows the results are the allocator's smallest blocks, of which others may be handed out.
@pytest.mark.gpu
@pytest.mark.parametrize("name", [n for n in NAMES if n != "token_logprobs of few rows"])
def test_results_take_no_memory_of_the_current_stream(name, monkeypatch):
    monkeypatch.setattr(base, "calls", calls)
    base.test_results_take_no_memory_of_the_current_stream(name)
