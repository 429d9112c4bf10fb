"""Plain 64-bit forms of the block operators, straight from their formulas and sequential over time, with
the error each output may have.

Bounds are counted in units of rounding: U32 = 2^-24 relative per fp32 operation, and half a step of
the output's type (2^-8 for bf16) for its rounding."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def offsets(lens):
    return [0] + torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist() if lens else [0]


def scan(gate, x, bias, h_in, lens, dy=None, dh_out=None):
    """gate, x, dy: [T, D] on the CPU, the sequences of `lens` one after another.  Returns a dict of the
    outputs and, under "tol", how far each may be off before its own rounding.

    A step is h = keep h + z x.  z and keep come from one exponential (relative error of e^-|u|: the
    product with log2 e is off by U32 |u| log2 e, times ln 2: |u| U32, and 4 more units for the exponential
    itself), a sum and a reciprocal (2 units each with the final product): z is off by at most
    (|u| + 10) U32, and keep by 6 U32 + z (|u| + 10) U32, whichever is the smaller one.  With H the
    largest |x|, |h_in|, a step adds an error of at most H ((9 + z (2 |u| + 24)) U32), and an error
    dies away as the product of the keeps: over a run e <- keep e + that.  The tile's maps
    are composed instead of applied in order: 2 more units per composition, of which there are at most 8
    in a tile and one per tile of at least 64 tokens: 32 + 2 T / 64 units of H, everywhere."""
    t_all, d = x.shape
    g64, x64 = gate.double(), x.double()
    u = g64 + (0.0 if bias is None else bias.double())
    z, keep = torch.sigmoid(u), torch.sigmoid(-u)
    b = len(lens)
    h0 = torch.zeros(b, d, dtype=torch.float64) if h_in is None else h_in.double()
    top = torch.maximum(x64.abs().amax(0) if t_all else torch.zeros(d, dtype=torch.float64),
                        h0.abs().amax(0) if b else torch.zeros(d, dtype=torch.float64))
    per_step = top * (9 + z * (2 * u.abs() + 24)) * U32
    flat = top * (32 + 2 * t_all / 64) * U32
    prev, h_all, err = torch.zeros(t_all, d).double(), torch.zeros(t_all, d).double(), torch.zeros(t_all, d).double()
    h_out, e_out = h0.clone(), torch.zeros(b, d).double()
    off = offsets(lens)
    for s in range(b):
        h, e = h0[s], torch.zeros(d, dtype=torch.float64)
        for t in range(off[s], off[s + 1]):
            prev[t] = h
            h = keep[t] * h + z[t] * x64[t]
            e = keep[t] * e + per_step[t]
            h_all[t], err[t] = h, e + flat
        if lens[s]:
            h_out[s], e_out[s] = h, e + flat
    out = {"y": h_all, "h_out": h_out, "tol": {"y": err, "h_out": e_out}}
    if dy is None:
        return out
    # backwards the same map with dy for x: an error of l_t is bounded by the run of |dy| the same way
    dy64 = dy.double()
    dh = torch.zeros(b, d, dtype=torch.float64) if dh_out is None else dh_out.double()
    dx, dg = torch.zeros(t_all, d).double(), torch.zeros(t_all, d).double()
    tx, tg = torch.zeros(t_all, d).double(), torch.zeros(t_all, d).double()
    dh_in, t_in = dh.clone(), torch.zeros(b, d).double()
    for s in range(b):
        G, size, e = dh[s], dh[s].abs(), torch.zeros(d, dtype=torch.float64)
        for t in reversed(range(off[s], off[s + 1])):
            lam, mag = dy64[t] + G, dy64[t].abs() + size          # mag bounds every |l_t| on the way
            rel = (9 + z[t] * (2 * u[t].abs() + 24)) * U32
            e_lam = e + mag * (34 + 2 * t_all / 64) * U32
            dx[t] = z[t] * lam
            tx[t] = z[t] * e_lam + (u[t].abs() + 12) * U32 * z[t] * mag
            f = z[t] * keep[t]
            dg[t] = f * (x64[t] - prev[t]) * lam
            wide = x64[t].abs() + prev[t].abs()
            tg[t] = f * (wide * e_lam + (err[t - 1] if t > off[s] else 0.0) * mag +
                         (2 * u[t].abs() + 24) * U32 * wide * mag)
            G, size, e = keep[t] * lam, keep[t] * mag, keep[t] * e + rel * mag
        dh_in[s] = G
        t_in[s] = e + size * (34 + 2 * t_all / 64) * U32
    out.update(dx=dx, dgate=dg, dh_in=dh_in, dbias=dg.sum(0))
    # the sum: 16 additions in a wave, 8 over waves, then T / 64 tiles (64 at a time) and 20 more
    out["tol"].update(dx=tx, dgate=tg, dh_in=t_in,
                      dbias=tg.sum(0) + dg.abs().sum(0) * (48 + t_all / 64 / 64) * U32)
    return out


# fp32 work of the norm on one row: at most 16 additions per thread, 6 in a wave, 16 over waves (half of
# it survives the square root), and 8 for the mean, eps, root, reciprocal and products
NORM_UNITS = 28


def rmsnorm(x, residual, weight, eps):
    """(r, n) in 64 bits; n is computed off by at most NORM_UNITS U32 |n|, r by U32 |r|."""
    r = x.double() + (0.0 if residual is None else residual.double())
    n = r / torch.sqrt(r.square().mean(-1, keepdim=True) + eps)
    return r, n * (1.0 if weight is None else weight.double())


def rmsnorm_backward(r, dy, weight, dr_out, eps):
    """dx, dweight in 64 bits and their bounds: each product and mean as in the forward pass (twice the
    units, three factors of the reciprocal root), dweight with the additions of its rows: every 64th
    row of a workgroup's and the workgroups' sums (at most rows / 256 + 64)."""
    r64, dy64 = r.double(), dy.double()
    rs = 1.0 / torch.sqrt(r64.square().mean(-1, keepdim=True) + eps)
    u = dy64 * (1.0 if weight is None else weight.double())
    a, c = rs * u, r64 * rs ** 3
    dx = a - c * (u * r64).mean(-1, keepdim=True)
    tol = (a.abs() + c.abs() * (u * r64).abs().mean(-1, keepdim=True)) * (3 * NORM_UNITS) * U32
    if dr_out is not None:
        dx = dx + dr_out.double()
        tol = tol + dx.abs() * U32
    term = dy64 * r64 * rs
    return dx, term.sum(0), tol, term.abs().sum(0) * (NORM_UNITS + r.shape[0] / 256 + 64) * U32


def assert_close(got, want, tol, what=""):
    """|got - want| <= tol + half a step of got's type, element by element."""
    g = got.detach().cpu()
    bound = tol + half_step(g.dtype) * (want.abs() + tol)
    bad = ~((g.double() - want).abs() <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3g at bound %.3g" % (
        what, int(bad.sum()), bad.numel(), float((g.double() - want).abs()[bad].max()), float(bound[bad].min()))
