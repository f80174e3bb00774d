"""MXFP4 tensors and the 4-bit projection on the GPU against their definition in 64 bits."""
import math

import pytest
import torch

import shape_adaptive_matrix_amd as sam
from tests import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(shape, dtype, seed, by=1.0):
    return (torch.randn(*shape, device="cuda", generator=gen(seed)) * by).to(TYPES[dtype])


def same_tensor(codes, scales, x):
    code, scale = ref.quantize(x)
    assert torch.equal(scales, scale)
    assert torch.equal(ref.unpack(codes), code)


SHAPES = [(1, 1), (1, 32), (3, 31), (2, 33), (5, 64), (7, 257), (130, 1000), (1, 8192), (33, 1025), (700, 96), (64, 4104)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize(shape, dtype):
    x = normal(shape, dtype, 3) * torch.exp(3 * torch.randn(shape[0], 1, device="cuda", generator=gen(4))).to(TYPES[dtype])
    x[:, ::7] = 0
    codes, scales = sam.quantize_mxfp4(x)
    same_tensor(codes, scales, x)
    ct, st = sam.quantize_mxfp4(x.t().contiguous(), trans=True)
    assert torch.equal(ct, codes) and torch.equal(st, scales)
    for out in TYPES.values():
        want = ref.values(ref.unpack(codes), scales, shape[1])
        got = sam.dequantize_mxfp4(codes, scales, shape[1], out_dtype=out)
        assert torch.equal(got, want.to(out))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_value(dtype):
    """Every 16-bit pattern, beside a largest value at several distances, Inf and NaN among them."""
    x = torch.arange(65536, device="cuda").to(torch.int16).view(TYPES[dtype])
    for big in (0.0, 6.0, 7.9375, 448.0):
        rows = torch.zeros(65536, 32, device="cuda", dtype=TYPES[dtype])
        rows[:, 5] = x
        rows[:, 9] = (x.float().abs() * big).to(TYPES[dtype])
        same_tensor(*sam.quantize_mxfp4(rows), rows)
        same_tensor(*sam.quantize_mxfp4(rows.t().contiguous(), trans=True), rows)


def test_float32_range():
    g = gen(8)
    bits = torch.randint(-2 ** 31, 2 ** 31 - 1, (4096, 64), device="cuda", generator=g, dtype=torch.int32)
    x = bits.view(torch.float32)
    x[:2048] = torch.where(torch.isfinite(x[:2048]), x[:2048], 1.0)
    x[7], x[8], x[9, 3] = 0.0, 1e-45, -math.inf
    # Values on and next to the borders between codes.
    y = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], device="cuda").repeat(8)
    near = torch.stack((y, torch.nextafter(y, y * 2), torch.nextafter(y, y * 0)))
    x[10:13] = near
    x[13:16] = -near * 2.0 ** -126
    same_tensor(*sam.quantize_mxfp4(x), x)
    same_tensor(*sam.quantize_mxfp4(x.t().contiguous(), trans=True), x)


def test_decode_every_code():
    codes = torch.arange(256, device="cuda").repeat_interleave(16).reshape(256, 16).to(torch.uint8)
    for first in range(0, 256, 32):
        scales = torch.arange(first, first + 32, device="cuda", dtype=torch.int32).to(torch.uint8).repeat(256, 1)
        wide = codes.repeat(1, 32)
        want = ref.values(ref.unpack(wide), scales, 1024)
        for out in TYPES.values():
            got = sam.dequantize_mxfp4(wide, scales, out_dtype=out)
            assert torch.equal(got.nan_to_num(nan=-1.25), want.to(out).nan_to_num(nan=-1.25))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,at", [(0, 1), (1, 0), (8, 0), (3, 2), (7, 5)])
def test_strides_and_alignment(pad, at, dtype):
    R, K = 37, 203
    whole = torch.full((R + 1, K + pad + at), math.nan, device="cuda").to(TYPES[dtype])
    x = whole[:R, at:at + K]
    x.copy_(normal((R, K), dtype, 5))
    codes, scales = sam.quantize_mxfp4(x)
    same_tensor(codes, scales, x)
    ct, st = sam.quantize_mxfp4(x, trans=True)
    same_tensor(ct, st, x.t())
    out = torch.full_like(whole, -7.0)
    sam.dequantize_mxfp4(codes, scales, K, X=out[:R, at:at + K])
    assert torch.equal(out[:R, at:at + K].double(), ref.values(ref.unpack(codes), scales, K))
    assert (out[R] == -7).all() and (out[:, :at] == -7).all() and (out[:, at + K:] == -7).all()


def test_large_tensor():
    """More than 2^31 values, offsets past 32 bits."""
    R, K = 66000, 32800
    x = torch.empty(R, K, device="cuda", dtype=torch.bfloat16)
    x.normal_(generator=gen(6))
    codes, scales = sam.quantize_mxfp4(x)
    for r in (0, 1, 32768, 65471, R - 1):
        same_tensor(codes[r:r + 1], scales[r:r + 1], x[r:r + 1])
    back = sam.dequantize_mxfp4(codes, scales, K)
    for r in (0, 65471, R - 1):
        assert torch.equal(back[r:r + 1].double(), ref.values(ref.unpack(codes[r:r + 1]), scales[r:r + 1], K))


# (M, N, K): single rows and few, around every tile of 16 to 256, odd K and N.
PRODUCTS = [(1, 1, 1), (1, 16, 32), (1, 4096, 1024), (2, 33, 95), (3, 1000, 257), (4, 17, 4100), (5, 300, 640), (8, 129, 2048),
            (15, 64, 130), (16, 2050, 513), (17, 48, 1024), (31, 80, 96), (32, 513, 1536), (33, 31, 700), (48, 96, 2080),
            (63, 200, 320), (64, 1024, 1024), (65, 129, 225), (128, 300, 999), (257, 513, 1025), (600, 700, 512)]


def product_bound(xq, w):
    """The instruction adds exact products (6 x 6 with steps of 1/4) of a block's
    scale; sums are FP32: K additions at most, half a step each of the terms'
    absolute sum."""
    K = xq.shape[1]
    return 2.0 ** -24 * (K + 32) * (xq.abs() @ w.abs().t())


def weight(N, K, seed):
    w = torch.randn(N, K, device="cuda", generator=gen(seed)) * K ** -0.5
    codes, scales = sam.quantize_mxfp4(w)
    return codes, scales, ref.values(ref.unpack(codes), scales, K)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", PRODUCTS, ids=str)
def test_linear(shape, dtype):
    M, N, K = shape
    x = normal((M, K), dtype, 11)
    x[:, ::13] *= 9
    codes, scales, w = weight(N, K, 12)
    xq = ref.values(*ref.quantize(x), K)
    want, bound = xq @ w.t(), product_bound(xq, w)
    y = sam.linear_mxfp4(x, codes, scales)
    assert y.dtype == torch.float32
    ref.close(y, want, bound)
    again = sam.linear_mxfp4(x, codes, scales)
    assert torch.equal(y, again)
    ref.close(sam.linear_mxfp4(x, codes, scales, out_dtype=TYPES[dtype]), want, bound)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(1, 300, 70), (7, 65, 130), (40, 129, 515), (300, 140, 96)], ids=str)
def test_linear_strides(shape, dtype):
    M, N, K = shape
    codes, scales, w = weight(N, K, 13)
    for pad, at in ((0, 0), (5, 1), (8, 0)):
        whole = torch.full((M + 1, K + pad + at), math.nan, device="cuda").to(TYPES[dtype])
        x = whole[:M, at:at + K]
        x.copy_(normal((M, K), dtype, 14))
        xq = ref.values(*ref.quantize(x), K)
        for out in {torch.float32, TYPES[dtype]}:
            y = torch.full((M + 1, N + pad + at), -7.0, device="cuda", dtype=out)
            sam.linear_mxfp4(x, codes, scales, Y=y[:M, at:at + N])
            ref.close(y[:M, at:at + N], xq @ w.t(), product_bound(xq, w))
            assert (y[M] == -7).all() and (y[:, :at] == -7).all() and (y[:, at + N:] == -7).all()


# Few rows by what their codes take of LDS, up to none: one and two blocks of the weight, whole lines and not.
HELD = [(16, 90, 6000), (5, 40, 16384), (24, 50, 8192), (31, 48, 8000), (64, 130, 4000), (9, 33, 33000), (16, 4200, 32768),
        (32, 100, 11008), (17, 4128, 16401), (32, 4200, 9216)]


@pytest.mark.parametrize("shape", HELD, ids=str)
def test_linear_of_long_rows(shape):
    M, N, K = shape
    x = normal((M, K), "f16", 43)
    codes, scales, w = weight(N, K, 44)
    xq = ref.values(*ref.quantize(x), K)
    want, bound = xq @ w.t(), product_bound(xq, w)
    y = torch.full((M + 1, N), -7.0, device="cuda", dtype=torch.float16)
    sam.linear_mxfp4(x, codes, scales, Y=y[:M])
    ref.close(y[:M], want, bound)
    assert (y[M] == -7).all()
    ref.close(sam.linear_mxfp4(x, codes, scales), want, bound)


@pytest.mark.parametrize("M,N,K", [(70, 333, 4000), (150, 2051, 1500), (301, 515, 225), (1025, 130, 700)], ids=str)
def test_what_a_workspace_held(M, N, K):
    """Scales of NaN left behind in a workspace, also beside the last rows, reach no result."""
    codes, scales, w = weight(N, K, 45)
    x = normal((M, K), "bf16", 46)
    want = sam.linear_mxfp4(x, codes, scales)
    xq = ref.values(*ref.quantize(x), K)
    ref.close(want, xq @ w.t(), product_bound(xq, w))
    for left in (0, 255):
        workspace = torch.full((32 << 20,), left, device="cuda", dtype=torch.uint8)
        assert torch.equal(sam.linear_mxfp4(x, codes, scales, workspace=workspace), want)


@pytest.mark.parametrize("M,N,K", [(3, 77, 500), (40, 130, 2080), (70, 333, 4000), (150, 2051, 1500), (300, 515, 225)], ids=str)
def test_linear_places(M, N, K):
    """Scales at every byte of a word, results that start inside one, neighbours left alone."""
    codes, scales, w = weight(N, K, 41)
    x = normal((M, K), "bf16", 42)
    want = sam.linear_mxfp4(x, codes, scales)
    xq = ref.values(*ref.quantize(x), K)
    ref.close(want, xq @ w.t(), product_bound(xq, w))
    room = torch.full((scales.numel() + 8,), 255, device="cuda", dtype=torch.uint8)
    for at in (1, 2, 3):
        moved = room[at:at + scales.numel()].view_as(scales)
        moved.copy_(scales)
        assert torch.equal(sam.linear_mxfp4(x, codes, moved), want)
        for out in (torch.float32, torch.bfloat16):
            y = torch.full((M * N + 8,), 3.0, device="cuda", dtype=out)
            sam.linear_mxfp4(x, codes, moved, Y=y[at:at + M * N].view(M, N))
            assert torch.equal(y[at:at + M * N].view(M, N), want.to(out))
            assert (y[:at] == 3).all() and (y[at + M * N:] == 3).all()
        room.fill_(255)


@pytest.mark.parametrize("M", [1, 4, 20, 70, 300])
def test_linear_nan_stays_in_its_row_and_column(M):
    N, K = 200, 160
    x = normal((M, K), "bf16", 15)
    codes, scales, w = weight(N, K, 16)
    clean = sam.linear_mxfp4(x, codes, scales)
    x[M // 2, 70] = math.inf
    scales[31, 1] = 255
    dirty = sam.linear_mxfp4(x, codes, scales)
    hit = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    hit[M // 2], hit[:, 31] = True, True
    assert dirty[hit].isnan().all() and torch.equal(dirty[~hit], clean[~hit])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 300, 200), (5, 64, 95), (33, 129, 513), (130, 96, 1000), (513, 300, 260)], ids=str)
def test_backward(shape, dtype):
    M, N, K = shape
    dy = normal((M, N), dtype, 21)
    codes, scales, w = weight(N, K, 22)
    want = dy.double() @ w
    # FP32 sums of exact products (FP32 dY: rounded ones), N of them, and split sums.
    bound = 2.0 ** -24 * (N + 64) * (dy.double().abs() @ w.abs())
    ref.close(sam.linear_mxfp4_backward(dy, codes, scales, K), want, bound)
    ref.close(sam.linear_mxfp4_backward(dy, codes, scales, K, out_dtype=TYPES[dtype]), want, bound)
    n = (K + 31) // 32 * 32
    wide = sam.linear_mxfp4_backward(dy, codes, scales)    # without K: whole blocks, zeros behind the weight
    assert wide.shape == (M, n) and not wide[:, K:].any()
    ref.close(wide[:, :K], want, bound)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_backward_strides(dtype):
    M, N, K = 37, 75, 130
    codes, scales, w = weight(N, K, 23)
    for pad in (0, 5, 8):
        whole = torch.full((M + 1, N + pad), math.nan, device="cuda").to(TYPES[dtype])
        whole[:M, :N] = normal((M, N), dtype, 24)
        dx = torch.full((M + 1, K + pad), -7.0, device="cuda").to(TYPES[dtype])
        sam.linear_mxfp4_backward(whole[:M, :N], codes, scales, dX=dx[:M, :K])
        dy = whole[:M, :N].double()
        ref.close(dx[:M, :K], dy @ w, 2.0 ** -24 * (N + 64) * (dy.abs() @ w.abs()))
        assert (dx[M] == -7).all() and (dx[:, K:] == -7).all()


def test_gradient_against_differences():
    """Where X lies on MXFP4 values and its changes do too, the projection is
    linear: differences give its gradient."""
    M, N, K = 3, 40, 64
    codes, scales, w = weight(N, K, 25)
    x = torch.randint(-6, 7, (M, K), device="cuda", generator=gen(26)).float()
    x[x.abs() == 5] = 4.0
    x[:, ::32] = 6.0                                     # every block's largest, so that its scale stays
    dy = normal((M, N), "f32", 27)
    grad = sam.linear_mxfp4_backward(dy, codes, scales, K)
    base = (sam.linear_mxfp4(x, codes, scales).double() * dy).sum()
    for k in (1, 33, 50):
        for m in range(M):
            y = x.clone()
            y[m, k] = 4.0 if x[m, k] != 4.0 else 2.0
            step = float(y[m, k] - x[m, k])
            diff = ((sam.linear_mxfp4(y, codes, scales).double() * dy).sum() - base) / step
            # FP32 rounding of N results on both sides.
            slack = 2.0 ** -23 * float((dy.double().abs() @ (w.abs() * 6).sum(1, keepdim=True)).max()) * (K + 32)
            assert abs(float(diff - grad[m, k])) <= slack


@pytest.mark.parametrize("M", [1, 8, 33, 200])
def test_captured_and_replayed(M):
    N, K = 320, 512
    codes, scales, w = weight(N, K, 31)
    x, dy = normal((M, K), "bf16", 32), normal((M, N), "bf16", 33)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            sam.linear_mxfp4_backward(sam.linear_mxfp4(x, codes, scales, out_dtype=torch.bfloat16), codes, scales, K)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = sam.quantize_mxfp4(x)
        y = sam.linear_mxfp4(x, codes, scales)
        dx = sam.linear_mxfp4_backward(dy, codes, scales, K)
    for seed in (34, 35, 36):
        x.copy_(normal((M, K), "bf16", seed))
        dy.copy_(normal((M, N), "bf16", seed + 9))
        want = sam.linear_mxfp4(x, codes, scales), sam.linear_mxfp4_backward(dy, codes, scales, K)
        qw = sam.quantize_mxfp4(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
        assert torch.equal(q[0], qw[0]) and torch.equal(q[1], qw[1])


def test_two_streams_at_once():
    N, K = 4096, 2048
    codes, scales, _ = weight(N, K, 41)
    xs = [normal((m, K), "bf16", 42 + m) for m in (1, 16, 64, 256)]
    want = [sam.linear_mxfp4(x, codes, scales) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [sam.linear_mxfp4(x, codes, scales, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)


def test_workspace_given():
    M, N, K = 40, 96, 128
    codes, scales, w = weight(N, K, 51)
    x = normal((M, K), "f16", 52)
    want = sam.linear_mxfp4(x, codes, scales)
    big = torch.full((1 << 22,), 0xAB, dtype=torch.uint8, device="cuda")
    assert torch.equal(sam.linear_mxfp4(x, codes, scales, workspace=big), want)
    with pytest.raises(sam.SamError):
        sam.linear_mxfp4(x, codes, scales, workspace=big[:64])
    with pytest.raises(sam.SamError):
        sam.linear_mxfp4_backward(want.half(), codes, scales, K, workspace=big[:64])
