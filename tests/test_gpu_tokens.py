"""Token log probabilities on the GPU against their definition in 64 bits."""
import math

import pytest
import torch

import shape_adaptive_matrix_amd as sam
from tests import tokens_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# (rows, V, top): rows of every length of a workgroup's turn, few rows (which
# are cut over workgroups) and many, odd lengths, fewer values than threads.
SHAPES = [(1, 1, 1), (3, 5, 5), (2, 130, 128), (300, 100, 20), (300, 1000, 128), (257, 4099, 3), (1, 4096, 0), (5, 20000, 64),
          (300, 8192, 0), (300, 8192, 5), (16, 32768, 64), (260, 33333, 20), (1, 131072, 20), (7, 131071, 128), (40, 50003, 1),
          (300, 66000, 128), (2, 1000003, 128), (600, 40000, 1)]


def make(R, V, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(R, V, device="cuda", generator=g) * 3
    t = torch.randint(V, (R,), device="cuda", generator=g).to(torch.int32)
    u = torch.randn(R, device="cuda", generator=g)
    v = torch.randn(R, device="cuda", generator=g)
    return z.to(TYPES[dtype]), t, u, v


def check(z, t, u, v, T, top, what=""):
    want = ref.reference(z, t, T, top, u, v)
    got = dict(zip(("logprob", "entropy", "norm", "top_logprob", "top_index"), sam.token_logprobs(z, t, T, top)))
    if top:
        assert torch.equal(got["top_index"], want["top_index"]), what
    for name in got:
        if name != "top_index":
            ref.close(got[name], want[name], f"{what} {name}")
    grad = sam.token_logprobs_grad(z, t, got["norm"], got["entropy"], u, v, T)
    ref.close(grad, want["grad"], what + " grad")
    return got, grad


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_against_definition(shape, dtype):
    R, V, top = shape
    for T in (1.0, 0.6, 3.0) if R * V < 1 << 24 else (0.8,):
        z, t, u, v = make(R, V, dtype, 3)
        t[1::5], t[2::11] = -1, V
        u[3::7] = 0.0
        v[3::14] = 0.0
        check(z, t, u, v, T, top, f"T={T}")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V", [300, 5001, 40000])
def test_masks_and_empty_rows(V, dtype):
    z, t, u, v = make(12, V, dtype, 5)
    z[0] = -math.inf                              # nothing left
    z[1] = -math.inf                              # one left
    z[1, V - 1] = 1.5
    z[2, ::2] = -math.inf
    z[3, 7:] = -math.inf                          # fewer than the alternatives asked for
    t[4] = 9
    z[4, 9] = -math.inf                           # the token is masked
    z[5] = torch.finfo(TYPES[dtype]).min          # the type's lowest value everywhere
    z[6, ::2] = torch.finfo(TYPES[dtype]).min
    z[7] = torch.finfo(TYPES[dtype]).max
    z[8, 1:] = 0.0                                # ties, both zeros
    z[8, ::3] = -0.0
    z[9] = 30000.0
    u[10], v[10] = 0.0, 0.0
    z[11] = z[11] / 100 + 1000                    # far from zero
    got, grad = check(z, t, u, v, 1.5, 20)
    assert got["top_index"][5].tolist() == list(range(20)) and got["top_index"][0].tolist() == list(range(20))
    assert got["logprob"][4] == -math.inf and got["entropy"][0] == 0 and got["entropy"][1] == 0
    assert not grad[0].any() and not grad[10].any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R,V", [(6, 5000), (300, 5000), (6, 70001), (300, 40000)])
def test_nan_and_inf_stay_in_their_row(R, V, dtype):
    z, t, u, v = make(R, V, dtype, 6)
    u[4] = v[4] = 0.0
    clean = sam.token_logprobs(z, t, 1.0, 16)
    cg = sam.token_logprobs_grad(z, t, clean[2], clean[1], u, v)
    z[1, 77], z[2, V - 1], z[3], z[4, 3] = math.nan, math.inf, math.nan, math.nan
    dirty = sam.token_logprobs(z, t, 1.0, 16)
    dg = sam.token_logprobs_grad(z, t, dirty[2], dirty[1], u, v)
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[1:5] = False
    for a, b in zip((*clean, cg), (*dirty, dg)):
        assert torch.equal(a[keep], b[keep])
    for r in (1, 2, 3, 4):
        assert dirty[0][r].isnan() and dirty[1][r].isnan() and dirty[2][r, 1].isnan() and dirty[3][r].isnan().all()
    assert torch.equal(dirty[4][1:5], ref.order(z[1:5])[:, :16].to(torch.int32))
    assert dg[1:4].isnan().any(1).all() and not dg[4].any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R", [2, 300])
def test_orders_that_cost_most(R, dtype):
    """Rising, falling, constant and repeated values, and the largest ones in one place."""
    V = 34000
    ramp = torch.arange(V, device="cuda").float() / V * 40 - 20
    for row in (ramp, ramp.flip(0), torch.zeros(V, device="cuda"), (torch.arange(V, device="cuda") % 7).float()):
        for top in (1, 20, 128):
            z = row.to(TYPES[dtype]).repeat(R, 1)
            z[1, 17000:17400] += 60
            z[1, 33990:] += 61
            got = sam.token_logprobs(z, torch.zeros(R, dtype=torch.int32, device="cuda"), 1.0, top)
            want = ref.reference(z[:2], torch.zeros(2, dtype=torch.int32, device="cuda"), 1.0, top)
            assert torch.equal(got[4][:2], want["top_index"])
            ref.close(got[3][:2], want["top_logprob"])
            ref.close(got[1][:2], want["entropy"])
            for x in got:
                assert torch.equal(x[2:], x[:1].expand_as(x[2:]))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R,V,pad", [(5, 4096, 8), (300, 1003, 6), (5, 1003, 5), (3, 140001, 3), (270, 33001, 1)])
def test_strides_places_and_alignment(R, V, pad, dtype):
    z, t, u, v = make(R, V, dtype, 8)
    zp = torch.full((R, V + pad), math.nan, device="cuda").to(z.dtype)
    gp = torch.full((R + 1, V + pad + 1), -7.0, device="cuda").to(z.dtype)
    zv, gv = zp[:, 1:V + 1], gp[:R, :V]
    zv.copy_(z)
    want = ref.reference(z, t, 1.0, 9, u, v)
    got = sam.token_logprobs(zv, t, 1.0, 9)
    for x, name in zip(got, ("logprob", "entropy", "norm", "top_logprob")):
        ref.close(x, want[name], name)
    assert torch.equal(got[4], want["top_index"])
    sam.token_logprobs_grad(zv, t, got[2], got[1], u, v, grad=gv)
    ref.close(gv, want["grad"])
    assert (gp[:, V:] == -7).all() and (gp[R] == -7).all()
    there = zv.clone()
    in_place = sam.token_logprobs_grad(there, t, got[2], got[1], u, v, grad=there)
    assert in_place is there and torch.equal(there, sam.token_logprobs_grad(zv.clone(), t, got[2], got[1], u, v))
    sam.token_logprobs_grad(zv, t, got[2], got[1], u, v, grad=zv)
    ref.close(zv, want["grad"])
    assert zp[:, 0].isnan().all() and zp[:, V + 1:].isnan().all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_parts_of_the_gradient(dtype):
    z, t, u, v = make(20, 3000, dtype, 9)
    logprob, entropy, norm = sam.token_logprobs(z, t, 0.9)
    for a, b in ((u, None), (None, v), (u, v)):
        want = ref.reference(z, t, 0.9, 0, a, b)["grad"]
        ref.close(sam.token_logprobs_grad(z, t, norm, entropy if b is not None else None, a, b, 0.9), want)
    assert not sam.token_logprobs_grad(z, t, norm).any()


def test_gradient_against_differences():
    z, t, u, v = make(4, 40, "f32", 10)
    T = 0.8
    logprob, entropy, norm = sam.token_logprobs(z, t, T)
    grad = sam.token_logprobs_grad(z, t, norm, entropy, u, v, T)
    h = 2.0 ** -7
    for j in range(40):
        step = torch.zeros_like(z)
        step[:, j] = h
        a, b = sam.token_logprobs(z + step, t, T), sam.token_logprobs(z - step, t, T)
        diff = (u * (a[0] - b[0]) + v * (a[1] - b[1])) / (2 * h)
        # The third derivative's part, (h / T)^2 times numbers of the size of p
        # times (log p)^2, at most 4 here, and FP32 results (2^-24 of values up
        # to 32, over 2 h).
        slack = (u.abs() + v.abs()) * ((h / T) ** 2 * 4 / T + 2.0 ** -24 * 32 * 8 / (2 * h))
        assert ((diff - grad[:, j]).abs() <= slack).all()


@pytest.mark.parametrize("R,V", [(1, 131072), (20, 50000), (300, 9000)])
def test_same_bits_captured_and_replayed(R, V):
    z, t, u, v = make(R, V, "bf16", 11)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            sam.token_logprobs(z, t, 1.0, 8)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sam.token_logprobs(z, t, 1.0, 8)
        grad = sam.token_logprobs_grad(z, t, got[2], got[1], u, v)
    for seed in (12, 13, 14):
        z.copy_(make(R, V, "bf16", seed)[0])
        want = sam.token_logprobs(z, t, 1.0, 8)
        wg = sam.token_logprobs_grad(z, t, want[2], want[1], u, v)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*got, grad), (*want, wg)):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    zs = [make(R, V, "bf16", 20 + R) for R, V in ((1, 131072), (16, 131072), (300, 30000), (2, 9001))]
    want = [sam.token_logprobs(z, t, 1.0, 20) for z, t, _, _ in zs]
    streams = [torch.cuda.Stream() for _ in zs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [sam.token_logprobs(z, t, 1.0, 20, stream=s) for (z, t, _, _), s in zip(zs, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_alternatives_feed_the_distillation():
    """A teacher's most likely entries as the distillation takes them: the loss of the teacher against itself, over all
    its entries, is zero."""
    z, t, _, _ = make(50, 96, "f32", 30)
    best, index = sam.token_logprobs(z, t, 1.0, 96)[3:]
    loss, grad = sam.distill(z, best, index)
    # p log p and p log q cancel up to FP32 roundings of logs up to 32.
    assert float(loss.abs().max()) <= 2.0 ** -24 * 32 * 16 and float(grad.abs().max()) <= 2.0 ** -24 * 64


def test_large_offsets():
    """Rows past 2^31 values."""
    R, V = 17000, 131072
    z = torch.empty(R, V, device="cuda", dtype=torch.bfloat16)
    z.normal_(generator=torch.Generator(device="cuda").manual_seed(40))
    t = torch.arange(R, device="cuda", dtype=torch.int32)
    u, v = torch.ones(R, device="cuda"), torch.ones(R, device="cuda")
    got = sam.token_logprobs(z, t, 1.0, 4)
    rows = torch.tensor([0, 16383, 16384, R - 1], device="cuda")
    keep = z[rows].clone()
    sam.token_logprobs_grad(z, t, got[2], got[1], u, v, grad=z)
    want = ref.reference(keep, t[rows], 1.0, 4, u[rows], v[rows])
    for x, name in zip(got, ("logprob", "entropy", "norm", "top_logprob")):
        ref.close(x[rows], want[name], name)
    assert torch.equal(got[4][rows], want["top_index"])
    ref.close(z[rows], want["grad"])
