"""Distillation loss on the GPU against its definition in 64 bits."""
import math

import pytest
import torch

import shape_adaptive_matrix_amd as sam
from tests import distill_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# (rows, V, top): each length of row that stays in registers at 256, 512 and
# 1024 threads, with many and with few rows, rows that pass registers and LDS
# (fp32 only: over 114688 values), odd lengths (rows then start anywhere),
# vocabularies shorter than a piece, more entries than threads.
SHAPES = [(1, 1, 1), (3, 5, 2), (7, 130, 130), (300, 1000, 8), (300, 4099, 20), (300, 8192, 33), (20, 32768, 16),
          (300, 20000, 64), (260, 33333, 7), (270, 65536, 12), (5, 131072, 300), (3, 200001, 1024)]


def make(R, V, k, dtype, seed, t_dtype=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = (torch.randn(R, V, device="cuda", generator=g) * 3).to(TYPES[dtype])
    t = (torch.randn(R, k, device="cuda", generator=g) * 4).to(TYPES[t_dtype or dtype])
    idx = torch.rand(R, V, device="cuda", generator=g).topk(k, dim=1).indices.to(torch.int32)
    w = torch.rand(R, device="cuda", generator=g) + 0.25
    return z, t, idx, w


def check(z, t, idx, w, T, what=""):
    want = ref.reference(z, t, idx, w, T)
    before = z.clone()
    loss, lse = sam.distill_loss(z, t, idx, w, T)
    both, grad = sam.distill(z, t, idx, w, T)
    later = sam.distill_grad(z, lse, t, idx, w, T)
    assert torch.equal(z.view(torch.int16 if z.element_size() == 2 else torch.int32),
                       before.view(torch.int16 if z.element_size() == 2 else torch.int32))
    ref.close(loss, *want[0], what + " loss")
    ref.close(both, *want[0], what + " loss with gradient")
    ref.close(lse, *want[1], what + " lse")
    ref.close(grad, *want[2], what + " gradient with loss")
    ref.close(later, *want[2], what + " gradient")
    return loss, lse, grad, later


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_against_definition(shape, dtype):
    for i, (T, t_dtype) in enumerate(((1.0, dtype), (2.5, "f32"), (0.7, "bf16"))):
        z, t, idx, w = make(*shape, dtype, 31 + i, t_dtype)
        w[1::7] = 0.0
        idx[2::9] = -1
        idx[:, ::5] = torch.where(torch.arange(shape[0], device="cuda")[:, None] % 2 == 0, idx[:, ::5], shape[1] + 3)
        check(z, t, idx, w if i else None, T, f"T={T}")


@pytest.mark.parametrize("dtype", list(TYPES))
def test_masks_and_empty_rows(dtype):
    z, t, idx, w = make(12, 3001, 9, dtype, 5)
    ninf = -math.inf
    z[0] = ninf                               # no logit left
    z[1, :3000] = ninf                        # one left
    idx[1] = 3000
    t[2], idx[3], w[4] = ninf, -1, 0.0        # no teacher, no entries, no weight
    z[5, idx[5, 0].item()] = ninf             # the teacher wants a masked entry: loss inf
    t[6, 1] = ninf
    z[6, idx[6, 1].item()] = ninf             # ... but not with p = 0
    z[7] = torch.finfo(TYPES[dtype]).min      # a mask of the type's lowest value, everywhere
    z[8, ::2] = torch.finfo(TYPES[dtype]).min
    loss, lse, grad, later = check(z, t, idx, w, 1.5)
    assert loss[5] == math.inf and lse[0] == ninf
    for row in (0, 2, 3, 4):
        assert loss[row] == 0 and not grad[row].any() and not later[row].any()
    assert not grad[5].isnan().any()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_nan_stays_in_its_row(dtype):
    z, t, idx, w = make(9, 5000, 6, dtype, 6)
    clean = [*sam.distill_loss(z, t, idx, w), *sam.distill(z, t, idx, w)]
    z[2, 77], z[3, 4999], t[5, 1], idx[5, 1] = math.nan, math.inf, math.nan, 8
    z[6, 5] = math.nan
    w[6] = 0.0
    dirty = [*sam.distill_loss(z, t, idx, w), *sam.distill(z, t, idx, w)]
    keep = torch.tensor([0, 1, 4, 7, 8], device="cuda")
    for a, b in zip(clean, dirty):
        assert torch.equal(a[keep], b[keep])
    for row in (2, 3, 5):
        assert dirty[0][row].isnan() and dirty[2][row].isnan()
    assert dirty[3][2].isnan().all() and dirty[0][6] == 0 and dirty[2][6] == 0 and not dirty[3][6].any()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_entries_with_the_same_index_add_up(dtype):
    z, t, idx, w = make(40, 700, 24, dtype, 7)
    idx[:, 5:] = idx[:, 3:4]
    idx[::2, 1] = idx[::2, 0]
    check(z, t, idx, w, 1.25)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V,pad", [(4096, 8), (1003, 6), (1003, 5), (140001, 3)])
def test_strides_places_and_alignment(V, pad, dtype):
    z, t, idx, w = make(6, V, 10, dtype, 8)
    zp = torch.full((6, V + pad), math.nan, device="cuda").to(z.dtype)
    gp = torch.full((7, V + pad + 1), -7.0, device="cuda").to(z.dtype)
    zv, gv = zp[:, 1:V + 1], gp[:6, :V]
    zv.copy_(z)
    want = ref.reference(z, t, idx, w, 1.0)
    loss, _ = sam.distill(zv, t, idx, w, grad=gv)     # rows of the two start at different alignments
    ref.close(loss, *want[0])
    ref.close(gv, *want[2])
    assert (gp[:, V:] == -7).all() and (gp[6] == -7).all()
    gp[:6, :V] = -7.0
    _, lse = sam.distill_loss(zv, t, idx, w)
    sam.distill_grad(zv, lse, t, idx, w, grad=gv)
    ref.close(gv, *want[2])
    assert (gp[:, V:] == -7).all() and (gp[6] == -7).all()
    # In the logits' place: the same bits.
    apart = sam.distill(zv, t, idx, w)
    apart_grad = sam.distill_grad(zv, lse, t, idx, w)
    copy = zp.clone()
    sam.distill(copy[:, 1:V + 1], t, idx, w, grad=copy[:, 1:V + 1])
    assert torch.equal(copy[:, 1:V + 1], apart[1]) and copy[:, 0].isnan().all()
    copy = zp.clone()
    sam.distill_grad(copy[:, 1:V + 1], lse, t, idx, w, grad=copy[:, 1:V + 1])
    assert torch.equal(copy[:, 1:V + 1], apart_grad)


@pytest.mark.parametrize("T", [2.0 ** -40, 2.0 ** 40])
def test_outermost_temperatures(T):
    """Nearest to an argmax, and nearest to equal probabilities: what the loss
    and its gradient tend to there, and no overflow on the way."""
    z, t, idx, w = make(5, 600, 4, "f32", 13)
    loss, lse = sam.distill_loss(z, t, idx, w, T)
    both, grad = sam.distill(z, t, idx, w, T)
    assert all(torch.isfinite(x).all() for x in (loss, lse, both, grad))
    if T < 1:
        top, best = z.argmax(1), idx.gather(1, t.argmax(1, keepdim=True).long())[:, 0].long()
        want = torch.zeros_like(z).scatter_add_(1, top[:, None], (w * T)[:, None])
        want.scatter_add_(1, best[:, None], -(w * T)[:, None])
    else:   # q = 1 / V, p = 1 / top, each off by its exponents' 8 / T and FP32 sums' steps
        want = torch.full_like(z, 1 / 600).scatter_add_(1, idx.long(), torch.full_like(t, -0.25)) * (w * T)[:, None]
    assert ((grad - want).abs() <= 2.0 ** -20 * (w * T)[:, None]).all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_workgroups_take_many_rows(dtype):
    """More rows than workgroups, so that each takes several: rows that are not
    trained on, empty and masked ones between the others, odd lengths."""
    for R, V, k in ((11000, 701, 70), (6000, 5003, 128), (3500, 1001, 129), (2300, 9001, 70), (1100, 20011, 70)):
        z, t, idx, w = make(R, V, k, dtype, 14)
        w[::3] = 0.0
        z[w == 0] = math.nan
        idx[1::5] = -1
        z[2::7] = torch.where(w[2::7, None] == 0, z[2::7], torch.full_like(z[2::7], -math.inf))
        idx[4::9, 30:60] = idx[4::9, :30]
        zz = torch.where(w[:, None] == 0, torch.zeros_like(z), z)     # the reference has no such rows
        want = ref.reference(zz, t, idx, w, 1.5)
        loss, grad = sam.distill(z, t, idx, w, 1.5)
        ref.close(loss, *want[0])
        ref.close(grad, *want[2])
        loss, lse = sam.distill_loss(z, t, idx, w, 1.5)
        ref.close(loss, *want[0])
        ref.close(sam.distill_grad(z, lse, t, idx, w, 1.5), *want[2])


@pytest.mark.parametrize("dtype", list(TYPES))
def test_entries_at_the_ends_of_strips(dtype):
    """The gradient from an lse cuts rows into strips of 512 pieces (of 256 in
    short rows): entries on the values around every cut and at a row's end,
    where values that fill no piece belong to the last strip."""
    e = 4 if dtype == "f32" else 8
    for pieces in (256, 512, 1024):
        for over in (-1, 0, 1, 3):
            V = pieces * e + over
            z, t, _, w = make(40, V + 8, 48, dtype, 15)
            at = torch.cat([torch.arange(V - 16, V), torch.arange(V // 2 - 16, V // 2 + 16)])
            idx = at.to(torch.int32).cuda().expand(40, 48).contiguous()
            for off in (0, 1, 5):     # rows start anywhere
                zv = z[:, off:off + V]
                loss, lse = sam.distill_loss(zv, t, idx, w)
                want = ref.reference(zv, t, idx, w, 1.0)
                for _ in range(3):
                    ref.close(sam.distill_grad(zv, lse, t, idx, w), *want[2], f"V={V} offset {off}")


def test_gradient_is_the_loss_difference():
    """Central differences of the loss in a random direction, step h: off by
    O(h^2) of the third derivative and by the loss's FP32 error over h."""
    z, t, idx, w = make(16, 777, 12, "f32", 9)
    g = torch.Generator(device="cuda").manual_seed(1)
    d = torch.randn(16, 777, device="cuda", generator=g)
    d /= d.norm(dim=1, keepdim=True)
    h, T = 2.0 ** -6, 1.5
    _, grad = sam.distill(z, t, idx, w, T)
    up, down = z + h * d, z - h * d
    want = (grad.double() * (up.double() - down.double())).sum(1) / (2 * h)
    got = (sam.distill_loss(up, t, idx, w, T)[0].double() - sam.distill_loss(down, t, idx, w, T)[0].double()) / (2 * h)
    # |third derivative| along a unit vector is at most w T^2 / T^3 (|d| <= 1, so the
    # third cumulant of d under q is at most 8 in size); FP32 error of two losses by the bound.
    bound = ref.reference(z, t, idx, w, T)[0][1]
    loss = sam.distill_loss(z, t, idx, w, T)[0].double().abs()
    allowed = w.double() / T * 8 * h * h / 6 + 2 * (bound * 1.1 + 2.0 ** -24 * loss * 1.1) / (2 * h) + 1e-6
    assert ((got - want).abs() <= allowed).all()


def test_streams_graphs_and_repeats():
    z, t, idx, w = make(64, 50003, 20, "bf16", 10)
    def call(s=None):
        loss, lse = sam.distill_loss(z, t, idx, w, stream=s)
        return loss, lse, sam.distill_grad(z, lse, t, idx, w, stream=s), *sam.distill(z, t, idx, w, stream=s)
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
        z.mul_(0.75)
        eager = call()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a, b), k


def test_far_rows():
    """Rows past 2^31 bytes of logits and gradient."""
    R, V = 9000, 131072
    z = torch.zeros(R, V, dtype=torch.bfloat16, device="cuda")
    some = torch.tensor([0, 8191, 8192, 8999], device="cuda")
    zs, t, idx, w = make(4, V, 16, "bf16", 11)
    z[some] = zs
    ta, ia = t.new_zeros(R, 16), torch.full((R, 16), -1, dtype=torch.int32, device="cuda")
    ta[some], ia[some] = t, idx
    wa = torch.zeros(R, device="cuda")
    wa[some] = w
    want = ref.reference(zs, t, idx, w, 1.0)
    loss, grad = sam.distill(z, ta, ia, wa)
    ref.close(loss[some], *want[0])
    ref.close(grad[some], *want[2])
    rest = torch.ones(R, dtype=torch.bool, device="cuda")
    rest[some] = False
    assert not grad[rest].any()
    loss, lse = sam.distill_loss(z, ta, ia, wa)
    ref.close(lse[some], *want[1])
    sam.distill_grad(z, lse, ta, ia, wa, grad=z)
    ref.close(z[some], *want[2])


# More entries than the workgroup's waves take at once (64 each): 256 threads
# up to V = 8192 in 16 bits (16384 with many rows), 512 threads up to 65536
# with many rows; more rows than workgroups in the last three.
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R,V,k", [(R, V, k) for R in (40, 600) for V in (700, 4096, 8192, 16000, 60000)
                                   for k in (257, 300, 513, 700, 1024)] + [(2300, 700, 1024), (2300, 4000, 300), (1600, 20011, 600)])
def test_many_entries_in_the_logits_place(R, V, k, dtype):
    """The same bits in the logits' place as apart from them, and those of the definition."""
    g = torch.Generator(device="cuda").manual_seed(R + V + k)
    z = (torch.randn(R, V, device="cuda", generator=g) * 3).to(TYPES[dtype])
    t = (torch.randn(R, k, device="cuda", generator=g) * 4).to(TYPES[dtype])
    idx = torch.randint(-1, V, (R, k), device="cuda", generator=g, dtype=torch.int32)   # some more than once
    w = torch.rand(R, device="cuda", generator=g) + 0.25
    w[1::7] = 0.0
    loss, grad = sam.distill(z, t, idx, w, 1.5)
    own, _ = sam.distill_loss(z, t, idx, w, 1.5)
    place = z.clone()
    loss_in_place, same = sam.distill(place, t, idx, w, 1.5, grad=place)
    assert same is place
    assert torch.equal(loss, loss_in_place) and torch.equal(grad, place)
    for rows in torch.arange(R, device="cuda").split(256):
        want = ref.reference(z[rows], t[rows], idx[rows], w[rows], 1.5)
        ref.close(loss[rows], *want[0], "loss with gradient")
        ref.close(own[rows], *want[0], "loss")
        ref.close(grad[rows], *want[2], "gradient")
