"""Results that a call makes itself belong to the stream that it runs on: the
memory of torch's current stream may still be in use there."""
import contextlib
import types

import pytest
import torch

import shape_adaptive_matrix_amd as sam

M, K, N, R, ADAPTERS, TOP = 1024, 512, 2048, 8, 3, 4


def calls(device):
    """(name, call of a stream) for every entry point that makes a result."""
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=device)  # noqa: E731
    X, W, A, B, dY = t(M, K), t(K, N), t(ADAPTERS, R, K), t(ADAPTERS, R, N), t(M, N)
    ids = torch.zeros(M, dtype=torch.int32, device=device)
    teacher, index = t(M, TOP), torch.zeros(M, TOP, dtype=torch.int32, device=device)
    lse = torch.zeros(M, device=device)
    mx = [torch.zeros(*s, dtype=torch.uint8, device=device) for s in ((M, K), (M, K // 32), (N, K), (N, K // 32))]
    return [
        ("gemm", lambda s: sam.gemm(X, W, stream=s)),
        ("gemm_noalloc", lambda s: sam.gemm_noalloc(X, W, stream=s)),
        ("gemm_ex", lambda s: sam.gemm_ex(X, W, stream=s)),
        ("gemm_mxfp8", lambda s: sam.gemm_mxfp8(*mx, stream=s)),
        ("adapter_gemm", lambda s: sam.adapter_gemm(X, W, A, B, ids, stream=s)),
        ("adapter_gemm of bf16", lambda s: sam.adapter_gemm(X, W, A, B, ids, out_dtype=X.dtype, stream=s)),
        ("adapter_backward", lambda s: sam.adapter_backward(dY, X, W, A, B, ids, stream=s)),
        ("distill_loss", lambda s: sam.distill_loss(dY, teacher, index, stream=s)),
        ("distill_grad", lambda s: sam.distill_grad(dY, lse, teacher, index, stream=s)),
        ("distill", lambda s: sam.distill(dY, teacher, index, stream=s)),
    ]


@pytest.mark.skipif(torch.cuda.is_available(), reason="host tensors: checks what is done without a GPU")
@pytest.mark.parametrize("name", [n for n, _ in calls("cpu")])
def test_results_are_allocated_on_the_stream(name, monkeypatch):
    call = dict(calls("cpu"))[name]
    inside, made = [], []
    empty, new_empty = torch.empty, torch.Tensor.new_empty

    @contextlib.contextmanager
    def on(stream):
        inside.append(stream)
        yield
        inside.pop()

    def recorded(make):
        def f(*a, **k):
            made.append(bool(inside))
            return make(*a, **k)
        return f

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", recorded(empty))
    monkeypatch.setattr(torch.Tensor, "new_empty", recorded(new_empty))
    monkeypatch.setattr(sam, "_on_device", lambda tensors, *a, **k: "cpu")
    monkeypatch.setattr(sam, "_one_gpu", lambda *a: 0)
    with pytest.raises(sam.SamError) as e:    # there is no GPU to run it on
        call(types.SimpleNamespace(cuda_stream=0))
    assert e.value.name == "SAM_ERR_UNSUPPORTED_DEVICE"
    assert made and all(made)


@pytest.mark.gpu
@pytest.mark.parametrize("name", [n for n, _ in calls("cpu")])
def test_results_take_no_memory_of_the_current_stream(name):
    """Blocks just freed on the current stream, where work may still be
    writing them, are not handed out for another stream's results."""
    call = dict(calls("cuda"))[name]
    like = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    tensors = [t for t in (like if isinstance(like, tuple) else (like,)) if t is not None]
    sizes = [(t.shape, t.dtype) for t in tensors]
    freed = [t.untyped_storage().data_ptr() for t in tensors]
    del like, tensors
    again = [torch.empty(s, dtype=d, device="cuda") for s, d in sizes]
    assert set(t.data_ptr() for t in again) & set(freed)   # what the current stream would get
    freed += [t.data_ptr() for t in again]
    del again
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    side.synchronize()
    for t in got if isinstance(got, tuple) else (got,):
        assert t.data_ptr() not in freed
