"""m3_rmsnorm and its backward pass against the formulas in 64 bits: every width class of the kernels
(rows on 16 lanes, on a wave, on a workgroup), odd widths and pitches, in-place outputs, 8-bit rows
and groups, rows of zeros, infinities and NaN.  Bounds: tests/block_ref.py."""
from __future__ import annotations

import pytest
import torch

from block_ref import NORM_UNITS, U32, assert_close, rmsnorm, rmsnorm_backward
from state_space_sequence_m3_amd import m3block

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
IO = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
SHAPES = [(1, 1), (3, 7), (5, 128), (2, 129), (37, 512), (1, 513), (9, 1000), (4, 1025), (6, 2048), (3, 2050), (5, 4096),
          (2, 4097), (3, 8192), (2, 8199), (3, 16384), (2, 16383), (1100, 96), (700, 640)]


def draw(n, d, io, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return r(n, d).to(io), (3 * r(n, d)).to(io), 1 + 0.2 * r(d), r(n, d).to(io), r(n, d).to(io)


def check_q(q, scale, n_ref, group):
    """scale = max |n| / 448 (one unit for the division), q within half a step of n / scale: 2^-4 relative,
    at least 2^-10 (half the smallest step), plus what n and scale are off by."""
    rows, d = n_ref.shape
    ng = 1 if group == 0 else -(-d // group)
    w = d if group == 0 else group
    pad = torch.nn.functional.pad(n_ref, (0, ng * w - d)).view(rows, ng, w)
    s_ref = pad.abs().amax(-1) / 448
    s_ref = torch.where(s_ref == 0, torch.ones_like(s_ref), s_ref)
    got = scale.cpu().double()
    assert got.shape == s_ref.shape
    assert ((got - s_ref).abs() <= (NORM_UNITS + 2) * U32 * s_ref).all()
    want = (pad / s_ref.unsqueeze(-1)).view(rows, -1)[:, :d]
    v = q.cpu().to(torch.float32).double()
    assert ((v - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10).double()) +
            (2 * NORM_UNITS + 6) * U32 * 448).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", SHAPES)
def test_forward(io, n, d):
    x, res, w, _, _ = draw(n, d, IO[io], n * 7 + d)
    r_ref, n_ref = rmsnorm(x, res, w, EPS)
    y, r, q, s = m3block.m3_rmsnorm(x.to(DEV), res.to(DEV), w.to(DEV), EPS, quant=True)
    torch.cuda.synchronize()
    assert_close(r, r_ref, r_ref.abs() * U32, "r")
    assert_close(y, n_ref, n_ref.abs() * NORM_UNITS * U32, "y")
    check_q(q, s, n_ref, 0)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("n,d", [(5, 31), (4, 100), (6, 128), (3, 300), (2, 1111), (3, 4096), (2, 12345)])
def test_groups(io, group, n, d):
    x, res, w, _, _ = draw(n, d, IO[io], d + group)
    _, n_ref = rmsnorm(x, None, w, EPS)
    y, r, q, s = m3block.m3_rmsnorm(x.to(DEV), None, w.to(DEV), EPS, want_y=False, quant=True, group=group)
    torch.cuda.synchronize()
    assert y is None and r is None
    check_q(q, s, n_ref, group)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", SHAPES)
def test_backward(io, n, d):
    _, r, w, dy, dr = draw(n, d, IO[io], n * 5 + d)
    dx_ref, dw_ref, t_dx, t_dw = rmsnorm_backward(r, dy, w, dr, EPS)
    dx, dw = m3block.m3_rmsnorm_backward(r.to(DEV), dy.to(DEV), w.to(DEV), dr.to(DEV), EPS)
    torch.cuda.synchronize()
    assert_close(dx, dx_ref, t_dx, "dx")
    assert_close(dw, dw_ref, t_dw, "dweight")
    dx_ref, _, t_dx, _ = rmsnorm_backward(r, dy, None, None, EPS)
    dx, dw = m3block.m3_rmsnorm_backward(r.to(DEV), dy.to(DEV), eps=EPS)
    torch.cuda.synchronize()
    assert dw is None
    assert_close(dx, dx_ref, t_dx, "dx without weight and dr")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [130, 4096, 4099])
def test_pitches_and_places(io, d):
    """Rows inside wider ones, at any element; r_out over the residual, y over x; dx over dr_out."""
    n = 9
    x, res, w, dy, dr = draw(n, d, IO[io], d)
    r_ref, n_ref = rmsnorm(x, res, w, EPS)
    wide = torch.full((n, 2 * d + 7), 5.0, dtype=IO[io], device=DEV)
    xs, rs = wide[:, 1:d + 1], wide[:, d + 4:2 * d + 4]
    xs.copy_(x), rs.copy_(res)
    y, r, _, _ = m3block.m3_rmsnorm(xs, rs, w.to(DEV), EPS, r_out=rs, y=xs)
    torch.cuda.synchronize()
    assert y is xs and r is rs
    assert_close(r, r_ref, r_ref.abs() * U32, "r")
    assert_close(y, n_ref, n_ref.abs() * NORM_UNITS * U32, "y")
    rest = torch.cat([wide[:, :1], wide[:, d + 1:d + 4], wide[:, 2 * d + 4:]], 1)
    assert (rest == 5.0).all()
    wide[:, 1:d + 1], wide[:, d + 4:2 * d + 4] = dy.to(DEV), dr.to(DEV)
    dx_ref, dw_ref, t_dx, t_dw = rmsnorm_backward(res, dy, w, dr, EPS)
    dx, dw = m3block.m3_rmsnorm_backward(res.to(DEV), xs, w.to(DEV), rs, EPS, dx=rs)
    torch.cuda.synchronize()
    assert_close(dx, dx_ref, t_dx, "dx")
    assert_close(dw, dw_ref, t_dw, "dweight")
    dx, _ = m3block.m3_rmsnorm_backward(res.to(DEV), xs, w.to(DEV), dr.to(DEV), EPS, dx=xs)
    torch.cuda.synchronize()
    assert_close(dx, dx_ref, t_dx, "dx over dy")


def test_no_rows_and_leading_dimensions():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    y, r, q, s = m3block.m3_rmsnorm(e, e.clone(), quant=True)
    assert y.shape == (0, 64) and q.shape == (0, 64) and s.shape == (0, 1)
    dx, dw = m3block.m3_rmsnorm_backward(e, e.clone(), torch.ones(64, device=DEV))
    torch.cuda.synchronize()
    assert dx.shape == (0, 64) and not dw.any()
    x, _, w, _, _ = draw(12, 64, torch.float32, 1)
    a = m3block.m3_rmsnorm(x.view(3, 4, 64).to(DEV), weight=w.to(DEV), quant=True, group=32)
    b = m3block.m3_rmsnorm(x.to(DEV), weight=w.to(DEV), quant=True, group=32)
    torch.cuda.synchronize()
    assert a[0].shape == (3, 4, 64) and a[3].shape == (3, 4, 2)
    assert torch.equal(a[0].view(12, 64), b[0]) and torch.equal(a[3].view(12, 2), b[3])


@pytest.mark.parametrize("d", [64, 700, 4096, 9000])
def test_zero_infinite_and_nan_rows(d):
    x = torch.randn(6, d)
    x[1], x[2, 3], x[3, d - 1], x[4] = 0.0, float("nan"), float("inf"), x[4] * 1e-30
    y, _, q, s = m3block.m3_rmsnorm(x.to(DEV), quant=True, eps=0.0 if d == 64 else EPS)
    yg, _, qg, sg = m3block.m3_rmsnorm(x.to(DEV), quant=True, group=32, eps=EPS)
    torch.cuda.synchronize()
    q, qg = q.float(), qg.float()
    for row in (0, 5):
        assert torch.isfinite(y[row]).all() and torch.isfinite(q[row]).all()
    if d == 64:     # eps 0: a row of zeros is 0 / 0, a tiny one is as good as any other
        assert torch.isnan(y[1]).all() and torch.isnan(s[1]).all()
        ref = x[4].double() / x[4].double().square().mean().sqrt()
        # squares of 1e-30 are 0 in fp32
        assert torch.isinf(y[4]).all() or torch.allclose(y[4].cpu().double(), ref, rtol=1e-5)
    else:
        assert not y[1].any() and not q[1].any() and s[1] == 1.0
        # tiny rows: n = x / sqrt(eps), about 3e-28, scaled up to 448 by a scale of about 1e-30
        assert float(q[4].abs().max()) == 448.0
        assert float(qg[4].abs().max()) == 448.0
    assert torch.isnan(y[2]).all() and torch.isnan(q[2]).all() and torch.isnan(s[2])
    assert torch.isnan(qg[2]).all() and torch.isnan(sg[2]).all()
    # an infinity: r / inf = 0 elsewhere, inf / inf = NaN in its place, as the formula says
    assert torch.isnan(y[3, d - 1]) and not y[3, :d - 1].any()
    assert torch.isnan(s[3]) and torch.isnan(sg[3, -1])


def test_scales_near_the_smallest_numbers():
    """n so small that 1 / scale would overflow: q still is n / scale."""
    d = 64
    x = torch.randn(3, d)
    w = torch.full((d,), 1e-37)
    y, _, q, s = m3block.m3_rmsnorm(x.to(DEV), weight=w.to(DEV), quant=True, eps=EPS)
    torch.cuda.synchronize()
    n = y.cpu().double()
    v = q.float().cpu().double()
    want = n / s.cpu().double()
    assert torch.isfinite(v).all()
    # scale has about 2^-37 * 2^-9 * 2^149: at least 13 bits left, so 449 may round into 448
    assert ((v - want).abs() <= want.abs() * 2.0 ** -4 + 2.0 ** -10 + 0.1).all()


def test_equal_inputs_give_equal_bits():
    x, res, w, dy, dr = (v.to(DEV) for v in draw(3000, 768, torch.bfloat16, 5))
    first = m3block.m3_rmsnorm(x, res, w, quant=True) + m3block.m3_rmsnorm_backward(res, dy, w, dr)
    for _ in range(3):
        again = m3block.m3_rmsnorm(x, res, w, quant=True) + m3block.m3_rmsnorm_backward(res, dy, w, dr)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(first, again))


def test_gradient_against_differences():
    """Central differences of the 64-bit norm confirm the reference's gradients."""
    r, dy, w = torch.randn(3, 6).double(), torch.randn(3, 6).double(), torch.randn(6).double()
    dx, dw, _, _ = rmsnorm_backward(r, dy, w, None, EPS)
    loss = lambda r, w: float((rmsnorm(r, None, w, EPS)[1] * dy).sum())
    for v, g, f in ((r, dx, lambda e: loss(e, w)), (w, dw, lambda e: loss(r, e))):
        for i in range(v.numel()):
            up, down = v.clone(), v.clone()
            up.view(-1)[i] += 1e-6
            down.view(-1)[i] -= 1e-6
            assert abs((f(up) - f(down)) / 2e-6 - float(g.reshape(-1)[i])) < 1e-6


def test_rows_past_four_gigabytes():
    n, d, pitch = 2200, 256, 1 << 20
    x, res, w, dy, dr = draw(n, d, torch.bfloat16, 9)
    buf = torch.empty(n, pitch, dtype=torch.bfloat16, device=DEV)
    place = lambda o, v: buf[:, o:o + d].copy_(v)
    r_ref, n_ref = rmsnorm(x, res, w, EPS)
    y, r, q, s = m3block.m3_rmsnorm(place(0, x), place(300, res), w.to(DEV), EPS, quant=True, y=buf[:, 600:600 + d],
                                    r_out=buf[:, 900:900 + d])
    dx, dw = m3block.m3_rmsnorm_backward(place(1200, res), place(1500, dy), w.to(DEV), place(1800, dr), EPS,
                                         dx=buf[:, 2100:2100 + d])
    torch.cuda.synchronize()
    assert_close(r, r_ref, r_ref.abs() * U32, "r")
    assert_close(y, n_ref, n_ref.abs() * NORM_UNITS * U32, "y")
    check_q(q, s, n_ref, 0)
    dx_ref, dw_ref, t_dx, t_dw = rmsnorm_backward(res, dy, w, dr, EPS)
    assert_close(dx, dx_ref, t_dx, "dx")
    assert_close(dw, dw_ref, t_dw, "dweight")


def e4m3_values():
    """The values of codes 0 to 126: 0 to 448."""
    return torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("d", [64, 512, 1024, 2048, 16384])
def test_quotients_next_to_borders(d, group):
    """Rows of ones and eps 0 make n the weight itself (a power of two of squares sums to its number, whose mean is 1),
    so scale and q follow from fp32 divisions alone: q = round(n / scale) for quotients on the borders between two
    8-bit values and up to two units beside them, all equal."""
    g = torch.Generator().manual_seed(d + group)
    w = group or d
    top = (1 + torch.rand(d // w, 1, generator=g)) * 2.0 ** torch.randint(-20, 20, (d // w, 1), generator=g)
    scale = top / 448
    values = e4m3_values()
    borders = (values[1:] + values[:-1])[torch.randint(0, 126, (d // w, w), generator=g)] / 2
    n = (borders * scale).view(torch.int32) + torch.randint(-2, 3, (d // w, w), generator=g, dtype=torch.int32)
    n = n.view(torch.float32)
    n[:, w // 2] = top[:, 0]
    want = (n / scale).to(torch.float8_e4m3fn)
    n *= 1 - 2 * torch.randint(0, 2, n.shape, generator=g)
    y, _, q, s = m3block.m3_rmsnorm(torch.ones(5, d, device=DEV), weight=n.reshape(-1).to(DEV), quant=True, group=group,
                                    eps=0.0)
    torch.cuda.synchronize()
    for row in range(5):
        assert torch.equal(y[row].cpu(), n.reshape(-1))
        assert torch.equal(s[row].cpu(), scale[:, 0])
        assert torch.equal(q[row].cpu().float().abs(), want.float().reshape(-1))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size,eps", [(1e12, EPS), (1e14, EPS), (1e16, EPS), (1e17, EPS), (1e-12, 0.0), (1e-14, 0.0), (1e-16, 0.0),
                                      (1e-3, 0.0)])
@pytest.mark.parametrize("d", [96, 700, 1100])
def test_backward_of_large_and_small_rows(io, size, eps, d):
    """Rows whose squares fp32 still holds (1100 of 1e34, and 1e-32) have gradients as good as any others."""
    n = 7
    _, r, w, dy, _ = draw(n, d, IO[io], d)
    r = (r.float() / 3 * size).to(IO[io])
    dr = (torch.randn(n, d, generator=torch.Generator().manual_seed(3)) / size).to(IO[io])
    dx_ref, dw_ref, t_dx, t_dw = rmsnorm_backward(r, dy, w, dr, eps)
    dx, dw = m3block.m3_rmsnorm_backward(r.to(DEV), dy.to(DEV), w.to(DEV), dr.to(DEV), eps)
    torch.cuda.synchronize()
    assert_close(dx, dx_ref, t_dx, "dx")
    assert_close(dw, dw_ref, t_dw, "dweight")


@pytest.mark.parametrize("group", [0, 32])
def test_scales_that_vanish(group):
    """Rows of ones and eps 0: n is the weight, here of 1 to 2^23 of fp32's smallest steps.  The scale is the least
    number of steps whose 448-fold holds the maximum (a division of whole numbers), and q = round(n / scale)."""
    for most in (1, 2, 200, 447, 448, 449, 668, 671, 900, 6000, 6500, 65000, 3000001, 2 ** 23):
        g = torch.Generator().manual_seed(most)
        steps = torch.randint(0, most + 1, (64,), generator=g)
        steps[5], steps[40] = most, most
        n = steps.to(torch.int32).view(torch.float32)
        assert int(n.view(torch.int32).max()) == most
        y, _, q, s = m3block.m3_rmsnorm(torch.ones(3, 64, device=DEV), weight=n.to(DEV), quant=True, group=group, eps=0.0)
        torch.cuda.synchronize()
        unit = -(-most // 448)
        want = (steps.double() / unit).float().to(torch.float8_e4m3fn)
        for row in range(3):
            assert torch.equal(y[row].cpu().view(torch.int32), steps.to(torch.int32)), most
            assert (s[row].cpu().view(torch.int32) == unit).all(), most
            assert torch.equal(q[row].cpu().float(), want.float()), most


def same_bits(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", [(50003, 96), (15001, 300), (9001, 1000), (3001, 1111), (1601, 4096), (700, 9001)])
def test_several_rows_to_a_workgroup(io, n, d):
    """Two rows or more to every workgroup and a ragged last round, in each layout of rows: every row against the
    formulas, the same in place, and the weight's gradient over all rows."""
    x, res, w, dy, dr = draw(n, d, IO[io], n + d)
    r_ref, n_ref = rmsnorm(x, res, w, EPS)
    xs, rs, wd = x.to(DEV), res.to(DEV), w.to(DEV)
    y, r, q, s = m3block.m3_rmsnorm(xs, rs, wd, EPS, quant=True)
    y2, r2, q2, s2 = m3block.m3_rmsnorm(xs, rs, wd, EPS, quant=True, group=32, r_out=rs, y=xs)
    torch.cuda.synchronize()
    assert_close(r, r_ref, r_ref.abs() * U32, "r")
    assert_close(y, n_ref, n_ref.abs() * NORM_UNITS * U32, "y")
    check_q(q, s, n_ref, 0)
    check_q(q2, s2, n_ref, 32)
    assert same_bits(y, y2) and same_bits(r, r2)
    dx_ref, dw_ref, t_dx, t_dw = rmsnorm_backward(res, dy, w, dr, EPS)
    rs, dys, drs = res.to(DEV), dy.to(DEV), dr.to(DEV)
    dx, dw = m3block.m3_rmsnorm_backward(rs, dys, wd, drs, EPS)
    e = dys.clone()
    over_dy, dw2 = m3block.m3_rmsnorm_backward(rs, e, wd, drs, EPS, dx=e)
    over_dr, dw3 = m3block.m3_rmsnorm_backward(rs, dys, wd, drs, EPS, dx=drs)
    torch.cuda.synchronize()
    assert_close(dx, dx_ref, t_dx, "dx")
    assert_close(dw, dw_ref, t_dw, "dweight")
    assert same_bits(dx, over_dy) and same_bits(dx, over_dr) and same_bits(dw, dw2) and same_bits(dw, dw3)


@pytest.mark.parametrize("io,n,d", [("f32", 4099, 4096), ("bf16", 8209, 4096), ("f32", 15203, 1111), ("bf16", 33203, 1013),
                                    ("f32", 250501, 67)])
def test_outputs_past_the_caches(io, n, d):
    """More than 256 MB moved, where outputs are stored non-temporally: 300 rows, first and last ones among them,
    against the formulas, and the weight's gradient over all rows."""
    es = 4 if io == "f32" else 2
    assert 4 * es * n * d > 1 << 28
    g = torch.Generator(device=DEV).manual_seed(n)
    x, res, dy, dr = (torch.randn(n, d, generator=g, device=DEV).mul_(k).to(IO[io]) for k in (1, 3, 1, 1))
    w = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
    pick = torch.cat([torch.arange(100, device=DEV), torch.randint(0, n, (100,), generator=g, device=DEV),
                      torch.arange(n - 100, n, device=DEV)])
    r_ref, n_ref = rmsnorm(x[pick].cpu(), res[pick].cpu(), w.cpu(), EPS)
    y, r, q, s = m3block.m3_rmsnorm(x, res, w, EPS, quant=True)
    torch.cuda.synchronize()
    assert_close(r[pick], r_ref, r_ref.abs() * U32, "r")
    assert_close(y[pick], n_ref, n_ref.abs() * NORM_UNITS * U32, "y")
    check_q(q.view(torch.uint8)[pick].view(torch.float8_e4m3fn), s[pick], n_ref, 0)
    del x, y, r, q
    dx, dw = m3block.m3_rmsnorm_backward(res, dy, w, dr, EPS)
    dx_ref, _, t_dx, _ = rmsnorm_backward(res[pick].cpu(), dy[pick].cpu(), w.cpu(), dr[pick].cpu(), EPS)
    _, dw_ref, _, t_dw = rmsnorm_backward(res, dy, w, None, EPS)
    torch.cuda.synchronize()
    assert_close(dx[pick], dx_ref, t_dx, "dx")
    assert_close(dw, dw_ref.cpu(), t_dw.cpu(), "dweight")
