"""Adapter projection on the GPU against its definition in 64 bits, with
element-wise bounds from the sums' lengths and the types' half steps."""
import pytest
import torch

import shape_adaptive_matrix_amd as sam
from tests import adapter_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}

# (M, K, N, rank, adapters): one row; every narrow tile; partials over one and
# several K ranges; ranks that fill no block of 16 and more than 64; rows that
# are no whole 16-byte pieces; short K (whole tiles with the term inside), the
# last two of them on 256 x 256 and 192 x 256 tiles.
SHAPES = [(1, 64, 64, 1, 1), (1, 4096, 512, 16, 4), (5, 200, 136, 8, 3), (16, 1, 1, 3, 2), (17, 264, 260, 4, 5),
          (33, 1000, 300, 24, 2), (64, 512, 1032, 16, 40), (100, 777, 333, 12, 7), (300, 130, 515, 64, 3),
          (129, 256, 640, 128, 2), (257, 2048, 384, 33, 3), (300, 2056, 8200, 48, 5), (4096, 64, 4096, 16, 8),
          (2049, 72, 4097, 40, 5)]


def make(M, K, N, r, n, dtype, seed, trans_w=False, runs=True):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    t = lambda *s, by=1.0: (torch.randn(*s, generator=g) * by).to(dt).cuda()  # noqa: E731
    X, W = t(M, K), t(*((N, K) if trans_w else (K, N)), by=K ** -0.5)
    A, B = t(n, r, K, by=K ** -0.5), t(n, r, N, by=r ** -0.5)
    ids = torch.randint(0, n, (M,), generator=g, dtype=torch.int32)
    if runs and M > 8:   # sequences of one request, and single rows of others in between
        seq = torch.sort(torch.randint(-1, n, (M,), generator=g, dtype=torch.int32)).values
        ids = torch.where(torch.rand(M, generator=g) < 0.9, seq, ids)
    for i, v in enumerate((-1, n, -7, 2 ** 31 - 1)):   # all of them: no adapter
        ids[3 + 5 * i::29] = v
    scale = torch.rand(n, generator=g).cuda() * 2 - 0.5
    return X, W, A, B, ids.cuda(), scale


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype):
    for i, (trans_w, out) in enumerate(((False, None), (True, TYPES[dtype]))):
        X, W, A, B, ids, scale = make(*shape, dtype, 11 + i, trans_w, runs=i == 0)
        Y = sam.adapter_gemm(X, W, A, B, ids, scale, trans_w=trans_w, out_dtype=out)
        assert Y.dtype == (out or torch.float32)
        ref.close(Y, *ref.forward(X, W, A, B, ids, scale, trans_w), f"trans_w={trans_w}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, dtype):
    M, K, N, r, n = shape
    for i, (trans_w, out) in enumerate(((False, TYPES[dtype]), (True, None))):
        X, W, A, B, ids, scale = make(*shape, dtype, 23 + i, trans_w, runs=i == 0)
        dY = (torch.randn(M, N, generator=torch.Generator().manual_seed(5)) * 0.1).to(X.dtype).cuda()
        got = sam.adapter_backward(dY, X, W, A, B, ids, scale, trans_w=trans_w, out_dtype=out)
        want = ref.backward(dY, X, W, A, B, ids, scale, trans_w)
        for g, w, name in zip(got, want, ("dX", "dA", "dB")):
            ref.close(g, *w, f"{name} trans_w={trans_w}")


# One adapter with hundreds of chunks of rows; T in one K range for both
# gradients; more adapters than a workgroup lists at a time, some with two
# chunks; whole tiles over a longer K.
MANY = [(20000, 64, 72, 8, 1), (33000, 136, 64, 24, 3), (20000, 40, 24, 4, 300), (300, 1000, 2000, 16, 4)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", MANY, ids=str)
def test_many_rows_chunks_and_adapters(shape, dtype):
    M, K, N, r, n = shape
    for runs in (True, False):
        X, W, A, B, ids, scale = make(*shape, dtype, 31 + runs, runs, runs)
        dY = (torch.randn(M, N, generator=torch.Generator().manual_seed(6)) * 0.1).to(X.dtype).cuda()
        Y = sam.adapter_gemm(X, W, A, B, ids, scale, trans_w=runs)
        ref.close(Y, *ref.forward(X, W, A, B, ids, scale, runs), f"Y runs={runs}")
        got = sam.adapter_backward(dY, X, W, A, B, ids, scale, trans_w=runs)
        for g, w, name in zip(got, ref.backward(dY, X, W, A, B, ids, scale, runs), ("dX", "dA", "dB")):
            ref.close(g, *w, f"{name} runs={runs}")


@pytest.mark.parametrize("M", [40, 2049])
def test_other_requests_inf_and_nan_stay_out(M):
    K, N, r, n = (2048, 384, 16, 6) if M == 40 else (72, 4097, 16, 6)
    X, W, A, B, ids, scale = make(M, K, N, r, n, "bf16", 3, runs=False)
    clean = sam.adapter_gemm(X, W, A, B, ids, scale)
    dY = torch.randn(M, N, device="cuda").to(X.dtype)
    clean_b = sam.adapter_backward(dY, X, W, A, B, ids, scale)
    A2, B2, s2 = A.clone(), B.clone(), scale.clone()
    A2[2], B2[2], B2[4, 0, 0], s2[5] = float("nan"), float("inf"), float("nan"), float("inf")
    dirty = sam.adapter_gemm(X, W, A2, B2, ids, s2)
    keep = (ids != 2) & (ids != 4) & (ids != 5)
    assert torch.equal(dirty[keep], clean[keep])
    assert not torch.isfinite(dirty[ids == 2]).any()
    dirty_b = sam.adapter_backward(dY, X, W, A2, B2, ids, s2)
    assert torch.equal(dirty_b[0][keep], clean_b[0][keep])
    for a in (0, 1, 3):
        assert torch.equal(dirty_b[1][a], clean_b[1][a]) and torch.equal(dirty_b[2][a], clean_b[2][a])


def test_inf_in_a_row_stays_in_it():
    X, W, A, B, ids, scale = make(50, 512, 256, 8, 3, "f16", 4, runs=False)
    clean = sam.adapter_gemm(X, W, A, B, ids, scale)
    X2 = X.clone()
    X2[7, 100], X2[20] = float("inf"), float("nan")
    dirty = sam.adapter_gemm(X2, W, A, B, ids, scale)
    keep = torch.ones(50, dtype=torch.bool, device="cuda")
    keep[7] = keep[20] = False
    assert torch.equal(dirty[keep], clean[keep])
    assert torch.isnan(dirty[20]).all()


@pytest.mark.parametrize("shape", [(9, 512, 256), (2049, 72, 4104)], ids=str)
def test_no_adapter_is_the_plain_projection(shape):
    M, K, N = shape
    X, W, A, B, ids, scale = make(M, K, N, 16, 3, "bf16", 6)
    none = torch.full_like(ids, -1)
    want = ref.forward(X, W, A, B, none, scale, False)
    Y = sam.adapter_gemm(X, W, A, B, none, scale)
    ref.close(Y, *want)
    assert torch.equal(Y, sam.adapter_gemm(X, W, A[:0], B[:0], ids))   # no adapters at all
    dY = torch.randn(M, N, device="cuda").to(X.dtype)
    dX, dA, dB = sam.adapter_backward(dY, X, W, A, B, none, scale)
    assert not dA.any() and not dB.any()
    ref.close(dX, *ref.forward(dY, W, B, A, none, scale, True))


def test_no_rows():
    X, W, A, B, ids, scale = make(1, 64, 72, 8, 3, "bf16", 6)
    assert sam.adapter_gemm(X[:0], W, A, B, ids[:0], scale).shape == (0, 72)
    dX, dA, dB = sam.adapter_backward(X.new_empty(0, 72), X[:0], W, A, B, ids[:0], scale,
                                      dA=torch.full((3, 8, 64), 7.0, device="cuda"))
    assert dX.shape == (0, 64) and not dA.any() and not dB.any()


@pytest.mark.parametrize("pad", [8, 3])
@pytest.mark.parametrize("shape", [(20, 512, 264, 16, 3), (1000, 128, 4000, 16, 3)], ids=str)
def test_views_with_padded_rows(shape, pad):
    M, K, N, r, n = shape
    X, W, A, B, ids, scale = make(*shape, "bf16", 8)
    nan = lambda rows, cols: torch.full((rows, cols), float("nan"), device="cuda").to(X.dtype)  # noqa: E731
    Xp, Wp, Yp = nan(M, K + pad), nan(K, N + pad), nan(M + 1, N + pad)
    Xp[:, :K], Wp[:, :N] = X, W
    Yp.fill_(-77.0)
    Y = sam.adapter_gemm(Xp[:, :K], Wp[:, :N], A, B, ids, scale, Y=Yp[:M, :N])
    ref.close(Y, *ref.forward(X, W, A, B, ids, scale, False))
    assert (Yp[:, N:] == -77.0).all() and (Yp[M] == -77.0).all()
    dY = torch.randn(M, N, device="cuda").to(X.dtype)
    dYp = nan(M, N + pad)
    dYp[:, :N] = dY
    dXp = torch.full((M + 1, K + pad), -77.0, device="cuda")
    sam.adapter_backward(dYp[:, :N], Xp[:, :K], Wp[:, :N], A, B, ids, scale, dX=dXp[:M, :K])
    ref.close(dXp[:M, :K], *ref.forward(dY, W, B, A, ids, scale, True))
    assert (dXp[:, K:] == -77.0).all() and (dXp[M] == -77.0).all()


@pytest.mark.parametrize("M", [7, 40, 300, 2049])
def test_w_with_padded_rows_is_read_in_place(M):
    """W's rows along the product's columns: what is behind a row is not looked at."""
    K, N = 520, 2501
    X, W, A, B, ids, scale = make(M, K, N, 16, 3, "bf16", 13)
    Wp = torch.full((K, 2504), float("nan"), device="cuda").to(X.dtype)
    Wp[:, :N] = W
    Y = sam.adapter_gemm(X, Wp[:, :N], A, B, ids, scale)
    ref.close(Y, *ref.forward(X, W, A, B, ids, scale, False))
    assert torch.equal(Y, sam.adapter_gemm(X, W, A, B, ids, scale))
    dY = torch.randn(M, K, device="cuda").to(X.dtype)   # of the projection onto W^T: dX = dY W
    Xt = torch.randn(M, N, device="cuda").to(X.dtype)
    got = sam.adapter_backward(dY, Xt, Wp[:, :N], B, A, ids, scale, trans_w=True)
    for g, w in zip(got, ref.backward(dY, Xt, W, B, A, ids, scale, True)):
        ref.close(g, *w)


def test_parts_of_the_backward_pass_alone():
    X, W, A, B, ids, scale = make(300, 264, 136, 16, 3, "bf16", 9)
    dY = torch.randn(300, 136, device="cuda").to(X.dtype)
    dX, dA, dB = sam.adapter_backward(dY, X, W, A, B, ids, scale)
    only = sam.adapter_backward(dY, X, W, A, B, ids, scale, need_dab=False)
    assert torch.equal(only[0], dX) and only[1] is None and only[2] is None
    only = sam.adapter_backward(dY, X, W, A, B, ids, scale, need_dx=False)
    assert only[0] is None and torch.equal(only[1], dA) and torch.equal(only[2], dB)


@pytest.mark.parametrize("M", [6, 700])
def test_gradients_are_the_differences_of_the_forward_pass(M):
    """Small integers make every product and sum exact, and Y is linear in
    each of X, A and B: central differences are exact too."""
    K, N, r, n = 96, 80, 8, 3
    g = torch.Generator().manual_seed(1)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    X, W, A, B, dY = ints(M, K), ints(K, N), ints(n, r, K), ints(n, r, N), ints(M, N)
    ids = torch.randint(-1, n, (M,), generator=g, dtype=torch.int32).cuda()
    scale = torch.tensor([1.0, 2.0, -1.0], device="cuda")
    grads = sam.adapter_backward(dY, X, W, A, B, ids, scale)
    for i, grad in enumerate(grads):
        d = ints(*grad.shape)
        ends = []
        for sign in (1, -1):
            args = [X, A, B]
            args[i] = (args[i] + sign * d).to(torch.bfloat16)
            Y = sam.adapter_gemm(args[0], W, args[1], args[2], ids, scale)
            ends.append(float((Y.double() * dY.double()).sum()))
        assert (ends[0] - ends[1]) / 2 == float((grad.double() * d.double()).sum()), ("X", "A", "B")[i]


@pytest.mark.parametrize("shape", [(24, 2048, 512, 16, 5), (2049, 256, 4096, 16, 5)], ids=str)
def test_streams_graphs_and_repeats(shape):
    X, W, A, B, ids, scale = make(*shape, "bf16", 12)
    dY = torch.randn(shape[0], shape[2], device="cuda").to(X.dtype)
    call = lambda s=None: (sam.adapter_gemm(X, W, A, B, ids, scale, stream=s),  # noqa: E731
                           *sam.adapter_backward(dY, X, W, A, B, ids, scale, stream=s))
    first = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(side)
    side.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = call()
    for k in range(3):
        X.add_(0.25)                     # eager work between the replays
        eager = call()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a, b), k


def test_far_rows():
    """Rows past 2^31 bytes of X, Y and dX."""
    M, K, N = 140000, 8192, 64
    X = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    some = torch.tensor([0, 1, 70001, 131071, 131072, 139999], device="cuda")
    g = torch.Generator().manual_seed(2)
    t = lambda *s, by=1.0: (torch.randn(*s, generator=g) * by).to(torch.bfloat16).cuda()  # noqa: E731
    X[some] = t(len(some), K)
    W, A, B = t(K, N, by=K ** -0.5), t(2, 16, K, by=K ** -0.5), t(2, 16, N, by=0.25)
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    ids[100000:] = 1
    Y = sam.adapter_gemm(X, W, A, B, ids, None, out_dtype=torch.bfloat16)
    ref.close(Y[some], *ref.forward(X[some], W, A, B, ids[some], None, False))
    left = torch.ones(M, dtype=torch.bool, device="cuda")
    left[some] = False
    assert not Y[left].any()
    dY = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    dY[some] = t(len(some), N)
    dX, dA, dB = sam.adapter_backward(dY, X, W, A, B, ids, None, out_dtype=torch.bfloat16)
    want = ref.backward(dY[some], X[some], W, A, B, ids[some], None, False)
    ref.close(dX[some], *want[0])
    assert not dX[left].any()
    ref.close(dA, *want[1])
    ref.close(dB, *want[2])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K,N", [(64, 72), (64, 512), (4096, 2049)])
def test_no_rows_over_any_length(K, N, dtype):
    X, W, A, B, ids, scale = make(1, K, N, 8, 3, dtype, 6)
    assert sam.adapter_gemm(X[:0], W, A, B, ids[:0], scale).shape == (0, N)
    for need_dx in (True, False):
        full = {name: torch.full((3, 8, c), 7.0, device="cuda") for name, c in (("dA", K), ("dB", N))}
        dX, dA, dB = sam.adapter_backward(X.new_empty(0, N), X[:0], W, A, B, ids[:0], scale, need_dx=need_dx, **full)
        assert (dX.shape == (0, K)) if need_dx else dX is None
        assert dA is full["dA"] and dB is full["dB"] and not dA.any() and not dB.any()


@pytest.mark.parametrize("K,N", [(520, 264), (777, 2049)])
def test_the_last_position_of_one_sequence(K, N):
    """One row with its sequence's stride, beyond what rows may be apart."""
    X, W, A, B, ids, scale = make(1, K, N, 16, 3, "bf16", 17)
    S = (1 << 21) // min(K, N) + 3
    ids.fill_(1)
    seq, dseq, out = (X.new_zeros(1, S, c) for c in (K, N, N))
    seq[:, -1], dseq[:, -1] = X, torch.randn(1, N, generator=torch.Generator().manual_seed(3)).to(X.dtype).cuda()
    if K % 8 == 0:   # operands start on 16 bytes
        Y = sam.adapter_gemm(seq[:, -1], W, A, B, ids, scale)
        assert torch.equal(Y, sam.adapter_gemm(X, W, A, B, ids, scale))
        ref.close(Y, *ref.forward(X, W, A, B, ids, scale, False))
        sam.adapter_gemm(X, W, A, B, ids, scale, Y=out[:, -1])
        assert torch.equal(out[:, -1], sam.adapter_gemm(X, W, A, B, ids, scale, out_dtype=X.dtype)) and not out[:, :-1].any()
        got = sam.adapter_backward(dseq[:, -1], seq[:, -1], W, A, B, ids, scale)
    else:
        wide = X.new_zeros(1, 1 << 22)
        wide[:, :K] = X
        got = sam.adapter_backward(dseq[:, -1].clone(), wide[:, :K], W, A, B, ids, scale)
    for g, w in zip(got, sam.adapter_backward(dseq[:, -1].clone(), X, W, A, B, ids, scale)):
        assert torch.equal(g, w)


def far_ranks(M, K, N, r, n, dtype, seed):
    """Small integers, each rank of A and B times a power of two of its own
    between 2^10 and 2^-14: T and the adapters' gradients are exact in FP32 (a
    rank's T are at most 2^10 multiples of its power), and the ranks' sizes
    are 24 bits apart."""
    g = torch.Generator().manual_seed(seed)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g).double()  # noqa: E731
    by = 2.0 ** torch.linspace(10, -14, r).round().double()[None, :, None]
    X, W, A, B, dY = ints(M, K), ints(K, N), ints(n, r, K) * by, ints(n, r, N) * by.flip(1), ints(M, N)
    ids = torch.randint(-1, n, (M,), generator=g, dtype=torch.int32).cuda()
    X, W, A, B, dY = (t.to(TYPES[dtype]).cuda() for t in (X, W, A, B, dY))
    return X, W, A, B, ids, torch.tensor([1.0, 2.0, -0.5], device="cuda")[:n], dY


def exact_gradients(X, W, A, B, ids, scale, dY):
    """dA and dB in 64 bits, where they are finite (the library's FP32 values exactly)."""
    (_, (dA, _), (dB, _)) = ref.backward(dY, X, W, A, B, ids, scale, False)
    return dA, dB


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(16, 96, 80, 8, 3), (100, 520, 264, 3, 2), (700, 96, 80, 24, 3), (5000, 200, 40, 40, 2),
                                   (3000, 72, 104, 128, 1)], ids=str)
def test_gradients_of_ranks_far_apart(shape, dtype):
    """A rank's gradient is as exact next to much larger ranks as alone."""
    args = far_ranks(*shape, dtype, 3)
    dA, dB = exact_gradients(*args)
    _, gA, gB = sam.adapter_backward(args[-1], *args[:-1])
    assert dA.abs().amax(2).min() > 0 and dB.abs().amax(2).min() > 0
    assert torch.equal(gA.double(), dA) and torch.equal(gB.double(), dB)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(40, 96, 80, 8, 3), (700, 96, 80, 24, 3), (5000, 200, 40, 40, 3)], ids=str)
def test_inf_and_nan_of_one_rank_stay_in_it(shape, dtype):
    """A's rank makes a row of dB Inf or NaN, B's a row of dA: the other ranks keep their bits."""
    X, W, A, B, ids, scale, dY = far_ranks(*shape, dtype, 4)
    dA, dB = exact_gradients(X, W, A, B, ids, scale, dY)
    A[1, 2, 5], B[2, 4, 7], A[2, 1, 0] = float("inf"), float("nan"), float("-inf")
    _, gA, gB = sam.adapter_backward(dY, X, W, A, B, ids, scale)
    for got, want, gone in ((gB, dB, [(1, 2), (2, 1)]), (gA, dA, [(2, 4)])):
        keep = torch.ones(want.shape[:2], dtype=torch.bool, device="cuda")
        for a, i in gone:
            keep[a, i] = False
            assert not torch.isfinite(got[a, i]).any()
        assert torch.equal(got[keep].double(), want[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_partials_stay_in_the_workspace(dtype):
    """As many adapters with two chunks as there can be (65 rows each), others
    with one or none, in a workspace of just the size that the library asks for."""
    M, K, N, r, n = 5000, 264, 136, 16, 90
    X, W, A, B, ids, scale = make(M, K, N, r, n, dtype, 19)
    g = torch.Generator().manual_seed(20)
    ids = (torch.arange(M, dtype=torch.int32) // 65)[torch.randperm(M, generator=g)].cuda()   # 77 adapters
    dY = torch.randn(M, N, generator=g).to(X.dtype).cuda()
    code = sam.BF16 if dtype == "bf16" else sam.F16
    need = sam._adapter_workspace_bytes("sam_adapter_backward_workspace", code, 0, M, N, K, n, r, N, K, N, 1, 1)
    whole = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    got = sam.adapter_backward(dY, X, W, A, B, ids, scale, workspace=whole[:need])
    for x, w, name in zip(got, ref.backward(dY, X, W, A, B, ids, scale, False), ("dX", "dA", "dB")):
        ref.close(x, *w, name)
    assert (whole[need:] == 77).all()
    assert not got[1][77:].any() and not got[2][77:].any()


# Split products (their partials added) and whole tiles with the term inside.
WHOLE = [(6, 64, 136, 8, 3), (20, 512, 264, 24, 2), (100, 264, 80, 16, 5), (300, 128, 520, 40, 3), (2100, 64, 264, 128, 2)]


def fits_two_values(t):
    """Whether rounding to two bfloat16 values would keep every one of t."""
    hi = t.to(torch.bfloat16).double()
    return torch.equal(hi + (t - hi).to(torch.bfloat16).double(), t)


def large_and_sparse(shape, dtype, seed):
    M, K, N, r, n = shape
    g = torch.Generator().manual_seed(seed)
    large = lambda *s: torch.randint(0, 128, s, generator=g).to(TYPES[dtype]).cuda()  # noqa: E731
    unit = lambda p, *s: ((torch.rand(*s, generator=g) < p) * (1 - 2 * torch.randint(0, 2, s, generator=g))).to(TYPES[dtype]).cuda()  # noqa: E731
    return large, unit, torch.randint(-1, n, (M,), generator=g, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", WHOLE, ids=str)
def test_fp32_results_take_the_intermediate_whole(shape, dtype):
    """T of 18 to 21 bits, and every sum exact in FP32: bfloat16 keeps T whole
    in an FP32 result, binary16 22 bits of the row's largest."""
    M, K, N, r, n = shape
    large, unit, ids = large_and_sparse(shape, dtype, 5)
    X, W, A = large(M, K), unit(0.5, K, N), large(n, r, K)
    B = torch.zeros(n, r, N, dtype=X.dtype, device="cuda")
    at = torch.arange(N, device="cuda")
    B[:, at % r, at] = 1 - 2 * (at // r % 2).to(X.dtype)     # a column takes one rank
    t = X.double() @ A[0].double().t()
    assert t.max() < 2 ** 22 and not fits_two_values(t)
    for trans_w in (False, True):
        Y = sam.adapter_gemm(X, W.t().contiguous() if trans_w else W, A, B, ids, trans_w=trans_w)
        want = ref.forward(X, W, A, B, ids, None, False)[0]
        assert want.abs().max() < 2 ** 24
        assert torch.equal(Y.double(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", WHOLE, ids=str)
def test_gradients_take_the_intermediate_whole(shape, dtype):
    """As above: T of X under dB, T of dY under dA."""
    M, K, N, r, n = shape
    large, unit, ids = large_and_sparse(shape, dtype, 6)
    W, A, B = unit(0.5, K, N), large(n, r, K), large(n, r, N)
    for X, dY, side in ((large(M, K), unit(2 / M, M, N), 2), (unit(2 / M, M, K), large(M, N), 1)):
        left, P, right = (X, A, dY) if side == 2 else (dY, B, X)
        t = left.double() @ P[0].double().t()
        assert t.max() < 2 ** 22 and not fits_two_values(t)
        assert (t.max() * right.double().abs().sum(0)).max() < 2 ** 24
        got = sam.adapter_backward(dY, X, W, A, B, ids, need_dx=False)
        assert torch.equal(got[side].double(), ref.backward(dY, X, W, A, B, ids, None, False)[side][0])


# Split products and whole tiles, narrow and wide.
@pytest.mark.parametrize("out", ["f32", "same"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(20, 512, 264, 8, 3), (40, 2048, 384, 40, 3), (300, 128, 520, 16, 3), (2049, 72, 4104, 16, 3)],
                         ids=str)
def test_inf_goes_where_the_formulas_take_it(shape, dtype, out):
    """Inf (NaN too, for parts of T are multiplied one by one) where the
    definition has Inf or NaN, and the other results' bits as without it."""
    M, K, N, r, n = shape
    X, W, A, B, ids, scale = make(M, K, N, r, n, dtype, 27, runs=False)
    ids[:n] = torch.arange(n, dtype=torch.int32)
    dY = (torch.randn(M, N, generator=torch.Generator().manual_seed(8)) * 0.1).to(X.dtype).cuda()
    to = X.dtype if out == "same" else None

    def results(X, A, B):
        return (sam.adapter_gemm(X, W, A, B, ids, scale, out_dtype=to),
                *sam.adapter_backward(dY, X, W, A, B, ids, scale, out_dtype=to))

    def check(got, clean, gone):
        for g, c, at, name in zip(got, clean, gone, ("Y", "dX", "dA", "dB")):
            lost = torch.zeros(g.shape, dtype=torch.bool, device="cuda")
            if at is not None:
                lost[at] = True
            assert not torch.isfinite(g[lost]).any(), name
            assert torch.equal(g[~lost], c[~lost]), name

    clean = results(X, A, B)
    assert all(torch.isfinite(c).all() for c in clean)
    mine = (ids == 1)[:, None]
    # A row of B: column 5 of its rows, and through dY B^T their dX and the rank's dA.
    B2, col, rank = B.clone(), torch.arange(N, device="cuda") == 5, torch.zeros(n, r, 1, dtype=torch.bool, device="cuda")
    B2[1, 2, 5], rank[1, 2] = float("inf"), True
    check(results(X, A, B2), clean, (mine & col, mine.expand(M, K), rank.expand(n, r, K), None))
    # A row of A: all of its rows of Y, column 5 of dX, the rank's dB.
    A2, col = A.clone(), torch.arange(K, device="cuda") == 5
    A2[1, 2, 5] = float("-inf")
    check(results(X, A2, B), clean, (mine.expand(M, N), mine & col, None, rank.expand(n, r, N)))
    # A row of X: its Y, column 5 of its adapter's dA, all of its dB.
    X2, whole = X.clone(), torch.zeros(n, 1, 1, dtype=torch.bool, device="cuda")
    X2[1, 5], whole[1] = float("inf"), True
    row = (torch.arange(M, device="cuda") == 1)[:, None]
    check(results(X2, A, B), clean, (row.expand(M, N), None, (whole & col).expand(n, r, K), whole.expand(n, r, N)))
