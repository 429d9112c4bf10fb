"""m3_grad_norm and m3_grad_clip against sums in 64 bits: one element to millions, many tensors, both
types, empty and unaligned ones, in place and not, coefficients of 1 and below, infinities and NaN."""
from __future__ import annotations

import ctypes

import pytest
import torch

from block_ref import U32, assert_close
from state_space_sequence_m3_amd import m3block

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def draw(sizes, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(torch.bfloat16 if i % 3 == 1 else torch.float32)
            for i, n in enumerate(sizes)]


def reference(grads, max_norm):
    norm = sum(t.double().square().sum() for t in grads if t.numel()).sqrt()
    return norm, torch.clamp(max_norm / (norm + 1e-6), max=1.0)


SIZES = [[1], [3, 0, 5], [16384], [16385, 1, 2047], [100003, 7, 64, 33000], [5] * 97, list(range(1, 260)), [0, 0, 9],
         [3000001, 100]]


@pytest.mark.parametrize("max_norm", [0.5, 1e9])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda v: "%dx%d" % (len(v), max(v)))
def test_clip(sizes, max_norm):
    """The sum is in fp64, so norm is one rounding off, coef two (norm is not rounded before it), and a
    scaled gradient two more and its own."""
    cpu = draw(sizes, len(sizes) + sizes[0])
    norm, coef = reference(cpu, max_norm)
    grads = [t.to(DEV) for t in cpu]
    stats = m3block.m3_grad_norm(grads, max_norm)
    out, stats2 = m3block.m3_grad_clip(grads, max_norm, out=[torch.full_like(t, 3.0) for t in grads])
    torch.cuda.synchronize()
    assert torch.equal(stats, stats2)
    assert abs(float(stats[0]) - float(norm)) <= 2 * U32 * float(norm)
    assert abs(float(stats[1]) - float(coef)) <= 2 * U32 * float(coef)
    for t, g, o in zip(cpu, grads, out):
        assert torch.equal(g.cpu(), t)                      # inputs untouched
        assert_close(o, t.double() * coef, (t.double() * coef).abs() * 3 * U32, "clipped")
    same, _ = m3block.m3_grad_clip(grads, max_norm)         # in place
    torch.cuda.synchronize()
    assert all(a is b for a, b in zip(same, grads))
    assert all(torch.equal(a, b) for a, b in zip(same, out))


def test_many_launches():
    """More tensors than one table holds, with more partial sums than the scaling pass adds itself."""
    sizes = [200000 + 13 * i for i in range(300)]
    grads = [torch.randn(n, device=DEV) for n in sizes]
    norm = sum(t.double().square().sum() for t in grads).sqrt()
    out, stats = m3block.m3_grad_clip(grads, 2.0, out=[torch.empty_like(t) for t in grads])
    torch.cuda.synchronize()
    coef = 2.0 / (norm + 1e-6)
    assert abs(float(stats[0]) - float(norm)) <= 2 * U32 * float(norm)
    for t, o in zip(grads, out):
        w = t.double() * coef
        assert ((o.double() - w).abs() <= 4 * U32 * w.abs()).all()


def test_unaligned_views():
    base = torch.randn(5000)
    flat = base.to(DEV)
    half = base.to(torch.bfloat16).to(DEV)
    grads = [flat[1:1000], flat[1001:4000], half[3:2000], half[2001:2002]]
    cpu = [t.cpu() for t in grads]
    norm, coef = reference(cpu, 1.0)
    m3block.m3_grad_clip(grads, 1.0)
    torch.cuda.synchronize()
    for t, o in zip(cpu, grads):
        assert_close(o, t.double() * coef, (t.double() * coef).abs() * 3 * U32, "clipped")
    for i in (0, 1000, 4000):
        assert flat[i].cpu() == base[i]
    assert torch.equal(half[:3].cpu(), base[:3].to(torch.bfloat16)) and half[2000].cpu() == base[2000].to(torch.bfloat16)


def test_large_and_small_magnitudes():
    """Squares beyond fp32's range in both directions."""
    for scale in (1e30, 1e-30):
        cpu = draw([1000, 500], 3, scale)
        norm, _ = reference(cpu, 1.0)
        stats = m3block.m3_grad_norm([t.to(DEV) for t in cpu])
        torch.cuda.synchronize()
        assert abs(float(stats[0]) - float(norm)) <= 2 * U32 * float(norm) and float(stats[1]) == 1.0


def test_non_finite_follows_the_formula():
    g = [torch.ones(100, device=DEV), torch.ones(50, device=DEV)]
    g[1][7] = float("inf")
    out, stats = m3block.m3_grad_clip(g, 1.0, out=[torch.empty_like(t) for t in g])
    torch.cuda.synchronize()
    assert torch.isinf(stats[0]) and stats[1] == 0.0 and not out[0].any() and torch.isnan(out[1][7])
    g[1][7] = float("nan")
    out, stats = m3block.m3_grad_clip(g, 1.0, out=[torch.empty_like(t) for t in g])
    torch.cuda.synchronize()
    assert torch.isnan(stats).all() and torch.isnan(out[0]).all()


def test_nothing_to_clip():
    _, stats = m3block.m3_grad_clip([], 1.0)
    _, stats2 = m3block.m3_grad_clip([torch.empty(0, device=DEV), None], 1.0)
    torch.cuda.synchronize()
    assert stats.tolist() == [0.0, 1.0] and stats2.tolist() == [0.0, 1.0]


def test_the_same_tensor_twice():
    t = torch.randn(1000, device=DEV)
    stats = m3block.m3_grad_norm([t, t])
    torch.cuda.synchronize()
    want = (2 * t.double().square().sum()).sqrt()
    assert abs(float(stats[0]) - float(want)) <= 2 * U32 * float(want)
    with pytest.raises(m3block.M3Error, match="M3_E_ALIAS"):
        m3block.m3_grad_clip([t, t], 1.0)


def test_more_elements_than_32_bits_count():
    """2^31 + 70001 bf16 elements of one tensor, all 0 but at its ends and around 2^31: norm sqrt(4 + 9 + 16 + 25 + 36),
    scaled to 1 (the sum is exact, the factor rounded to fp32, products to bf16: half a step and one unit)."""
    n = 2 ** 31 + 70001
    at = torch.tensor([0, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 65536, n - 1], device=DEV)
    v = torch.tensor([2.0, 3.0, 4.0, 5.0, 6.0], device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g[at] = v.bfloat16()
    stats = m3block.m3_grad_norm([g], 1.0)
    assert abs(float(stats[0]) - 90 ** 0.5) <= 90 ** 0.5 * 2.0 ** -23
    m3block.m3_grad_clip([g], 1.0)
    want = v.double() / (90 ** 0.5 + 1e-6)
    assert ((g[at].double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -22)).all()
    assert int(g.count_nonzero()) == 5


def test_equal_inputs_give_equal_bits():
    grads = [t.to(DEV) for t in draw([70001, 12, 900000], 8)]
    first = m3block.m3_grad_norm(grads)
    for _ in range(3):
        again = m3block.m3_grad_norm(grads)
        torch.cuda.synchronize()
        assert torch.equal(first, again)


def test_more_partial_sums_than_are_added_twice():
    """300 tensors of 15 units of 16384 elements make 4500 partial sums in four launches: over 4096 a launch of their
    own adds them, and all scaling passes take its sum."""
    grads = [torch.randn(230000 + 13 * i, device=DEV) for i in range(300)]
    table = (m3block.M3GradTensor * len(grads))()
    for t, g in zip(table, grads):
        t.src, t.dst, t.numel, t.io = g.data_ptr(), g.data_ptr(), g.numel(), m3block.M3_F32
    parts = m3block.load().m3_grad_workspace_bytes(ctypes.cast(table, ctypes.c_void_p), len(grads)) // 8 - 1
    assert parts > 4096
    norm = sum(t.double().square().sum() for t in grads).sqrt()
    coef = 2.0 / (norm + 1e-6)
    out, stats = m3block.m3_grad_clip(grads, 2.0, out=[torch.full_like(t, 3.0) for t in grads])
    alone = m3block.m3_grad_norm(grads, 2.0)
    want = [t.double() * coef for t in grads]
    m3block.m3_grad_clip(grads, 2.0)                        # in place
    torch.cuda.synchronize()
    assert torch.equal(stats, alone)
    assert abs(float(stats[0]) - float(norm)) <= 2 * U32 * float(norm)
    assert abs(float(stats[1]) - float(coef)) <= 2 * U32 * float(coef)
    for w, o, g in zip(want, out, grads):
        assert ((o.double() - w).abs() <= 4 * U32 * w.abs()).all()
        assert torch.equal(o, g)
