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


def confident(logits, T, u, v):
    """logprob of the largest entry, entropy, log of the sum, and the gradient there for that token, in float64, with
    bounds relative to what lies beside the largest entry: the others' sum r, not 1 + r."""
    T = float(torch.tensor(T, dtype=torch.float32))
    d = (logits.double() - logits.double().amax(1, keepdim=True)) / T
    e = torch.where(d < 0, torch.exp(d), 0.0)
    assert ((d == 0).sum(1) == 1).all()
    r, size = e.sum(1), torch.where(e > 0, -d, 0.0)
    D1, D2 = (e * size).sum(1), (e * size * size).sum(1)
    L = torch.log1p(r)
    H = L + D1 / (1 + r)
    # An exponent is off by 4 half steps of |d| (tokens_ref), 2^x by 4 more, a
    # sum by its chain of additions (a thread's values, joins); log1p, expm1 and the
    # last operations by a few.
    n = 64 + logits.shape[1] / 256
    br = ref.U32 * (4 * D1 + (4 + n) * r)
    bL = br + 4 * ref.U32 * L
    bH = bL + ref.U32 * (4 * D2 + (12 + n) * D1) + D1 * br + 4 * ref.U32 * H
    p = 1 / (1 + r)
    grad = (u.double() * r * p - v.double() * p * (H - L)) / T
    bound = (u.abs().double() * (2 * bL + 8 * ref.U32 * r) + v.abs().double() * (bL + bH + 8 * ref.U32 * H)) / T
    # 2^x under 2^-126 is 0: of V entries.
    tiny = 2.0 ** -126 * logits.shape[1]
    return {"logprob": (-L, bL + tiny), "entropy": (H, bH + 200 * tiny), "norm": (L, bL + tiny), "grad": (grad, bound + 200 * tiny)}


# Rows on a wave, on a workgroup, cut over several; V of a few pieces and of many.
# (bfloat16 values near 40 are 1/4 apart.)
@pytest.mark.parametrize("dtype,far", [("f32", 0.0), ("bf16", 0.0), ("f16", 0.0), ("f32", 40.0), ("f16", 40.0)])
@pytest.mark.parametrize("R,V,top", [(20, 900, 0), (20, 1003, 5), (600, 5001, 0), (300, 33333, 20), (270, 40000, 0), (2, 131075, 0),
                                     (3, 300000, 20), (1, 17, 3)], ids=str)
def test_confident_rows(R, V, top, dtype, far):
    """Rows with one entry of probability 1 - 1e-1 .. 1 - 1e-9: its log probability, the entropy, the norm and the gradient
    there are as exact as what lies beside it. far: a thread's sums by the other way, which values far from zero take."""
    g = torch.Generator(device="cuda").manual_seed(50)
    T = 0.9 if not far else 2.0 ** -9
    z = torch.randn(R, V, device="cuda", generator=g)
    at = torch.randint(V, (R,), device="cuda", generator=g)
    at[::7], at[1::7] = 0, V - 1                                  # the row's edges
    beside = 10.0 ** -(1 + 8 * torch.rand(R, device="cuda", generator=g))
    # In units of T; sum exp(z) of normal values is near V e^(1/2).
    z[torch.arange(R, device="cuda"), at] = torch.log(V * math.exp(0.5) / beside)
    z[::5, V // 3:V // 2] = -math.inf
    z[torch.arange(R, device="cuda"), at] = torch.log(V * math.exp(0.5) / beside)
    z = (z * T + far).to(TYPES[dtype])
    best = z.amax(1, keepdim=True)
    at = (z == best).to(torch.int8).argmax(1)
    if far:   # rounding near `far` may move an entry into the largest one's place
        z = torch.where((z == best) & (torch.arange(V, device="cuda") != at[:, None]), -math.inf, z)
    u = torch.randn(R, device="cuda", generator=g)
    v = 0.1 * torch.randn(R, device="cuda", generator=g)
    v[::2] = 0.0
    want = confident(z, T, u, v)
    tokens = at.to(torch.int32)
    got = sam.token_logprobs(z, tokens, T, top)
    for x, name in zip((got[0], got[1], got[2][:, 1]), ("logprob", "entropy", "norm")):
        ref.close(x, want[name], name)
    assert torch.equal(got[2][:, 0], best[:, 0].float())
    if top:
        assert torch.equal(got[4][:, 0], tokens) and torch.equal(got[3][:, 0], got[0])
    grad = sam.token_logprobs_grad(z, tokens, got[2], got[1], u, v, T)
    ref.close(grad.gather(1, at[:, None])[:, 0], want["grad"], "gradient at the token")
    check(z, tokens, u, v, T, top)                               # and everything else


@pytest.mark.parametrize("R,V,dtype", [(300, 262147, "f32"), (260, 1000003, "f32"), (257, 530001, "bf16"), (257, 530001, "f16")])
def test_long_rows_on_a_workgroup(R, V, dtype):
    """Rows so long that what a thread keeps stands for several turns' pieces: random, masked, constant, NaN."""
    z, t, u, v = make(R, V, dtype, 60)
    z[0], z[1], z[2, 7:] = -math.inf, 2.5, -math.inf
    z[3], z[4, ::2] = torch.arange(V, device="cuda") / V, -math.inf
    z[5], z[6] = -torch.arange(V, device="cuda") / V, torch.finfo(TYPES[dtype]).min
    z[7, V // 2:V // 2 + 300] += 40                              # the best next to each other
    z[8, 5], z[9, V - 1], z[10, V // 3] = math.nan, math.inf, math.nan
    rows = torch.cat((torch.arange(16, device="cuda"), torch.tensor([R // 2, R - 1], device="cuda")))
    for top in (20, 128):
        got = sam.token_logprobs(z, t, 1.0, top)
        want = ref.reference(z[rows], t[rows], 1.0, top)
        bad = torch.zeros(len(rows), dtype=torch.bool, device="cuda")
        bad[8:11] = True
        assert torch.equal(got[4][rows], want["top_index"])
        for x, name in zip(got, ("logprob", "entropy", "norm", "top_logprob")):
            a, b = want[name]
            ref.close(x[rows][~bad], (a[~bad], b[~bad]), name)
        assert got[0][8:11].isnan().all() and got[3][8:11].isnan().all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("top", [20, 128])
def test_candidates_of_many_parts(top, dtype):
    """Few rows cut over 64 workgroups, whose lists are joined: rising and falling rows, where almost every list's entries
    reach the bound, the best in one part, equal values, masked parts."""
    V = 1000003 if dtype == "f32" else 2000003
    ramp = (torch.arange(V, device="cuda").double() / V * 40 - 20).float()
    g = torch.Generator(device="cuda").manual_seed(61)
    noise = torch.randn(2, V, device="cuda", generator=g)
    one = noise[0].clone()
    one[V // 2:V // 2 + 5000] += 60
    masked = noise[1].clone()
    masked[: V // 4 * 3] = -math.inf
    rows = [ramp, ramp.flip(0), one, torch.zeros(V, device="cuda"), masked, torch.full((V,), -math.inf, device="cuda"), noise[0]]
    tokens = torch.tensor([V - 1, 0], dtype=torch.int32, device="cuda")
    for a, b in zip(rows, rows[1:] + rows[:1]):
        z = torch.stack((a, b)).to(TYPES[dtype])
        got = sam.token_logprobs(z, tokens, 1.0, top)
        want = ref.reference(z, tokens, 1.0, top)
        assert torch.equal(got[4], want["top_index"])
        for x, name in zip(got, ("logprob", "entropy", "norm", "top_logprob")):
            ref.close(x, want[name], name)
