"""Gradients of the first rows of sequences in bf16: a row that sees few keys has nearly all of dout . v_j - delta cancel, so
that a delta from the rounded output would leave its rounding whole.  Of rows that see at most 128 keys delta is the sum of
p_ij (dout_i . v_j) in fp32, and the bounds here are those of tests/attn_ref.py without the output's rounding."""
from __future__ import annotations

import pytest
import torch

import attn_ref
from block_ref import U32, assert_close, half_step
from state_space_sequence_m3_amd import m3attn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
FIRST = 128


def gradients(q, k, v, dout, lens):
    """dq, dk, dv [T, H, D] in 64 bits and their bounds."""
    io, hq, hk, d = q.dtype, q.shape[1], k.shape[1], q.shape[2]
    scale, h, group = d ** -0.5, half_step(q.dtype), hq // hk
    q, k, v, dout = (x.double() for x in (q, k, v, dout))
    out = {n: torch.zeros_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    tol = {n: torch.zeros_like(x) for n, x in out.items()}
    at = 0
    for n in lens:
        rows = slice(at, at + n)
        at += n
        seen = torch.ones(n, n, dtype=torch.bool).tril()
        for i in range(hq):
            j = i // group
            a = attn_ref.attend(q[rows, i], k[rows, j], v[rows, j], scale, seen, io)
            p, do = a["p"], dout[rows, i]
            rel = a["e"] + a["tol"]["lse"].unsqueeze(1)
            dp = do @ v[rows, j].T
            e_dp = d * U32 * (do.abs() @ v[rows, j].abs().T)
            delta = (p * dp).sum(1, keepdim=True)
            first = (p * (rel * dp.abs() + e_dp + (n + 16) * U32 * dp.abs())).sum(1, keepdim=True)
            later = (do.abs() * (a["tol"]["o"] + h * (a["o"].abs() + a["tol"]["o"]) + d * U32 * a["o"].abs())).sum(1, keepdim=True)
            e_delta = torch.where(torch.arange(n).unsqueeze(1) < FIRST, first, later)
            ds = p * (dp - delta)
            e_ds = p * (rel * (dp - delta).abs() + e_dp + e_delta + 3 * U32 * (dp.abs() + delta.abs()))
            e_ds = e_ds + (h + (n + 16) * U32) * (ds.abs() + e_ds)
            sums = (group * n + 16) * U32
            out["dq"][rows, i] = scale * (ds @ k[rows, j])
            tol["dq"][rows, i] = scale * (e_ds @ k[rows, j].abs())
            out["dk"][rows, j] += scale * (ds.T @ q[rows, i])
            tol["dk"][rows, j] += scale * ((e_ds + sums * ds.abs()).T @ q[rows, i].abs())
            out["dv"][rows, j] += p.T @ do
            tol["dv"][rows, j] += (p * (rel + h + sums)).T @ do.abs()
    return out, tol


def draw(t, hq, hk, d, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(t, h, d, generator=g).bfloat16() for h in (hq, hk, hk, hq)]


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("hq,hk,lens", [(4, 2, [1, 2, 0, 31, 32, 33, 64, 65]), (2, 2, [128, 1, 100, 129, 160]),
                                        (150, 150, [1, 33, 130]), (300, 100, [64, 127])])
def test_packed(hq, hk, lens, d):
    q, k, v, dout = draw(sum(lens), hq, hk, d, d)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    qd, kd, vd, dd = (x.to(DEV) for x in (q, k, v, dout))
    o, lse = m3attn.m3_attention(qd, kd, vd, cu, save_lse=True)
    g = m3attn.m3_attention_backward(qd, kd, vd, o, lse, dd, cu)
    torch.cuda.synchronize()
    want, tol = gradients(q, k, v, dout, lens)
    for x in "qkv":
        assert_close(g[x], want["d" + x], tol["d" + x], "d" + x)


@pytest.mark.parametrize("n", [1, 2, 40, 100, 150])
@pytest.mark.parametrize("hq,hk", [(2, 1), (320, 160)])
def test_dense(hq, hk, n):
    b, d = 2, 64
    q, k, v, dout = draw(b * n, hq, hk, d, n)
    qd, kd, vd, dd = (x.to(DEV).unflatten(0, (b, n)) for x in (q, k, v, dout))
    o, lse = m3attn.m3_attention(qd, kd, vd, save_lse=True)
    g = m3attn.m3_attention_backward(qd, kd, vd, o, lse, dd)
    torch.cuda.synchronize()
    want, tol = gradients(q, k, v, dout, [n] * b)
    for x in "qkv":
        assert_close(g[x].flatten(0, 1), want["d" + x], tol["d" + x], "d" + x)


@pytest.mark.parametrize("hq,hk", [(2, 1), (300, 100)])
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 14, 2.0 ** 18])
def test_one_token_of_large_scores(hq, hk, size):
    """One key alone: ds is 0 whatever the score.  p is off by |lse| 2^-23 of 1, below 2 here, delta by its quotient's and dp's
    rounding."""
    lens, d = [1] * 5, 64
    q, k, v, dout = draw(sum(lens), hq, hk, d, 3)
    big = size ** 0.5
    q, k = (q.float() * big).bfloat16(), (k.float() * big).bfloat16()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    qd, kd, vd, dd = (x.to(DEV) for x in (q, k, v, dout))
    o, lse = m3attn.m3_attention(qd, kd, vd, cu, save_lse=True)
    g = m3attn.m3_attention_backward(qd, kd, vd, o, lse, dd, cu)
    torch.cuda.synchronize()
    assert float(lse.abs().max()) > size / 8
    group, scale = hq // hk, d ** -0.5
    kg, vg = (x.double().repeat_interleave(group, 1) for x in (k, v))
    # dp in either kernel has an order of its own: d additions each, and 4 units of delta
    ds = 2 * (2 * d + 4) * U32 * (dout.double().abs() * vg.abs()).sum(-1, keepdim=True)
    assert (g["q"].cpu().double().abs() <= scale * ds * kg.abs() * (1 + half_step(torch.bfloat16)) ** 2).all()
    dk = (scale * ds * q.double().abs()).unflatten(1, (hk, group)).sum(2)
    assert (g["k"].cpu().double().abs() <= dk * (1 + half_step(torch.bfloat16)) ** 2).all()
