"""Plain 64-bit forms of the attention operators, straight from their formulas, with the error each output may
have.

Bounds are counted in units of rounding: U32 = 2^-24 relative per fp32 operation, and half a step of
a type (2^-8 for bf16) for each rounding to it."""
from __future__ import annotations

import torch

from block_ref import U32, half_step

NEG = float("-inf")


def score_error(q, k, scale, s):
    """How far a score may be off, in units of the exponent (q [n, D], k [m, D], s = scale q k^T, all 64 bits): D
    additions of the products, and the products with scale and log2 e, a subtraction of the row's maximum or lse and the
    exponential's argument: 6 more of the largest number there, which 4 maxima of |s| in the row and 40 bound."""
    size = scale * (q.abs() @ k.abs().T)
    top = s.abs().amax(1, keepdim=True) if s.shape[1] else s.abs()
    return (q.shape[1] * size + 6 * (s.abs() + 4 * top) + 40) * U32


def attend(q, k, v, scale, seen, io):
    """One head: q [n, D], k, v [m, D] 64 bits, seen [n, m].  Returns o, lse, p and their bounds under "tol"; rows that
    see nothing have o = 0 and lse = -inf.

    A probability is off by its score's error e, relative to itself, and rounded to io for its product with v (h); sums
    have at most m additions.  So o is off by sum p |v| (h + e + (m + 16) U32) for the numerator, and the
    same without h of |o| for the denominator."""
    n, m = q.shape[0], k.shape[0]
    s = scale * (q @ k.T)
    e = score_error(q, k, scale, torch.where(seen, s, torch.zeros_like(s)))
    s = torch.where(seen, s, torch.full_like(s, NEG))
    some = seen.any(1)
    lse = torch.where(some, torch.logsumexp(s, 1) if m else torch.full((n,), NEG).double(), torch.full((n,), NEG).double())
    p = torch.where(seen, torch.exp(s - torch.where(some, lse, torch.zeros_like(lse)).unsqueeze(1)), torch.zeros_like(s))
    h = half_step(io) if io is torch.bfloat16 else 0.0
    o = p @ v
    t_o = (p * (h + e + (m + 16) * U32)) @ v.abs() + o.abs() * (p * (e + (m + 16) * U32)).sum(1, keepdim=True)
    t_lse = (p * e).sum(1) + (m + 16 + 4 * torch.where(some, lse, torch.zeros_like(lse)).abs()) * U32
    return {"o": o, "lse": lse, "p": p, "e": e, "tol": {"o": t_o, "lse": t_lse}}


def prompt(q, k, v, lens, scale=None, dout=None):
    """Causal attention of packed q [T, Hq, D], k, v [T, Hkv, D] (io type, CPU) and, with dout, its gradients: a dict of
    outputs with their bounds under "tol".

    Backward: p is off by e and the error of lse; delta by what o is off (its bound and its rounding) times |dout|; dp by D
    additions.  ds then by p times that, and both p and ds are rounded to io for their products."""
    io, (t, hq, d), hk = q.dtype, q.shape, k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    h = half_step(io) if io is torch.bfloat16 else 0.0
    out = {"o": torch.zeros_like(q), "lse": torch.zeros(hq, t).double(), "tol": {"o": torch.zeros_like(q),
           "lse": torch.zeros(hq, t).double()}}
    if dout is not None:
        dout = dout.double()
        for name, like in (("dq", q), ("dk", k), ("dv", v)):
            out[name], out["tol"][name] = torch.zeros_like(like), torch.zeros_like(like)
    at = 0
    for n in lens:
        rows = slice(at, at + n)
        at += n
        if n == 0:
            continue
        seen = torch.ones(n, n, dtype=torch.bool).tril()
        for i in range(hq):
            j = i // (hq // hk)
            a = attend(q[rows, i], k[rows, j], v[rows, j], scale, seen, io)
            out["o"][rows, i], out["lse"][i, rows] = a["o"], a["lse"]
            out["tol"]["o"][rows, i], out["tol"]["lse"][i, rows] = a["tol"]["o"], a["tol"]["lse"]
            if dout is None:
                continue
            p, do = a["p"], dout[rows, i]
            rel = a["e"] + a["tol"]["lse"].unsqueeze(1)
            delta = (do * a["o"]).sum(1, keepdim=True)
            e_delta = (do.abs() * (a["tol"]["o"] + half_step(io) * (a["o"].abs() + a["tol"]["o"]) +
                                   d * U32 * a["o"].abs())).sum(1, keepdim=True)
            dp = do @ v[rows, j].T
            e_dp = d * U32 * (do.abs() @ v[rows, j].abs().T)
            ds = p * (dp - delta)
            e_ds = p * (rel * (dp - delta).abs() + e_dp + e_delta + 3 * U32 * (dp.abs() + delta.abs()))
            e_ds = e_ds + (h + (n + 16) * U32) * (ds.abs() + e_ds)
            out["dq"][rows, i] = scale * (ds @ k[rows, j])
            out["tol"]["dq"][rows, i] = scale * (e_ds @ k[rows, j].abs())
            group = (hq // hk) * n + 16
            out["dk"][rows, j] += scale * (ds.T @ q[rows, i])
            out["tol"]["dk"][rows, j] += scale * ((e_ds + group * U32 * ds.abs()).T @ q[rows, i].abs())
            out["dv"][rows, j] += p.T @ do
            out["tol"]["dv"][rows, j] += (p * (rel + h + group * U32)).T @ do.abs()
    return out


def rotate(x, pos, inv_freq, halves):
    """x [T, H, D] (io type) rotated at pos [T], 64 bits, and its bound: angles reduced to a turn are fp32 (half a unit of
    pi, 2 U32), sine and cosine 2 units each, two products and a sum."""
    r = 2 * inv_freq.shape[0]
    y = x.double().clone()
    tol = torch.zeros_like(y)
    ang = pos.double().unsqueeze(1) * inv_freq.double()
    cos, sin = ang.cos().unsqueeze(1), ang.sin().unsqueeze(1)
    a, b = (slice(0, r // 2), slice(r // 2, r)) if halves else (slice(0, r, 2), slice(1, r, 2))
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = u * cos - v * sin, u * sin + v * cos
    tol[..., a] = tol[..., b] = 8 * U32 * (u.abs() + v.abs())
    return y, tol


def step(q, keys, values, scale=None):
    """One token per sequence: q [b, Hq, D] (io type), keys and values lists of [Hkv, n, D].  Returns o, lse and bounds."""
    b, hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    o, lse, t_o, t_lse = (torch.zeros(b, hq, d).double(), torch.zeros(b, hq).double(), torch.zeros(b, hq, d).double(),
                          torch.zeros(b, hq).double())
    for s in range(b):
        hk, n = keys[s].shape[:2]
        for i in range(hq):
            j = i // (hq // hk)
            a = attend(q[s, i:i + 1].double(), keys[s][j].double(), values[s][j].double(), scale,
                       torch.ones(1, n, dtype=torch.bool), q.dtype)
            o[s, i], lse[s, i] = a["o"][0], a["lse"][0]
            t_o[s, i], t_lse[s, i] = a["tol"]["o"][0], a["tol"]["lse"][0]
    return {"o": o, "lse": lse, "tol": {"o": t_o, "lse": t_lse}}
