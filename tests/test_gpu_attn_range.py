"""Scores of any finite size, in m3_attention and m3_attention_step: up to the ends of fp32's range, all of a row far below or
above zero, equal and unequal ones.

Inputs make every score exact: queries have one element that is not zero, a power of two, and keys numbers of few
digits there, so the bounds hold no errors of scores.  A probability exp(s - max) is off by 2 |s - max| U32 (scale log2 e, and
its product with the score) and 16 U32 for the exponential; beyond differences of 200 it is zero in fp32."""
from __future__ import annotations

import pytest
import torch

from block_ref import U32, assert_close, half_step
from state_space_sequence_m3_amd import m3attn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
IO = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZES = [2.0 ** e for e in (20, 27, 28, 29, 31, 33, 40, 100, 126)]


def exact_inputs(n, hq, hk, d, io, size, sign, seed, scale):
    """q [n, Hq, D], k, v [n, Hkv, D]: scores are sign * size, or that times 127 / 128, key by key at random, and with a
    negative sign the first half of the keys all equal; the least size has up to 3 more."""
    g = torch.Generator().manual_seed(seed)
    q, k = torch.zeros(n, hq, d), torch.zeros(n, hk, d)
    less = torch.rand(n, hk, generator=g) < 0.5
    if sign < 0:
        less[:n // 2] = False
    q[:, :, 3] = 2.0 ** 60
    k[:, :, 3] = torch.where(less, 127.0 / 128, 1.0) * sign * size / scale / 2.0 ** 60
    if size == SIZES[0]:
        q[:, :, 5], k[:, :, 5] = 1.0, torch.randint(0, 4, (n, hk), generator=g) / scale
    v = torch.randn(n, hk, d, generator=g)
    q, k, v = q.to(io), k.to(io), v.to(io)
    at_first = (q[0, 0].double() @ k[0, 0].double()) * scale - sign * size * (127 / 128 if less[0, 0] else 1)
    assert 0 <= at_first <= (3 if size == SIZES[0] else 0)
    return q, k, v


def attend(q, k, v, scale, seen, io):
    """One head in 64 bits: o, lse and their bounds."""
    n = k.shape[0]
    s = torch.where(seen, scale * (q.double() @ k.double().T), torch.tensor(float("-inf")).double())
    top = s.amax(1, keepdim=True)
    p = torch.exp(s - top)
    rel = ((top - s).clamp(max=200) * 2 + 16 + n) * U32
    total = p.sum(1, keepdim=True)
    o = p @ v.double() / total
    h = half_step(io) if io is torch.bfloat16 else 0.0
    tol = (p * (h + rel)) @ v.double().abs() / total + o.abs() * (p * rel).sum(1, keepdim=True) / total
    lse = (top + total.log()).squeeze(1)
    return o, tol, lse, 4 * U32 * lse.abs() + 32 * U32 + (p * rel).sum(1) / total.squeeze(1)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("hq,hk,d,n", [(2, 1, 64, 300), (130, 2, 32, 300), (130, 2, 128, 200)])
def test_prompt_scores_far_from_zero(io, sign, hq, hk, d, n):
    io = IO[io]
    for i, size in enumerate(SIZES):
        for scale in (1.0, 2.0 ** -5):
            if size / scale > 2.0 ** 126:
                continue
            q, k, v = exact_inputs(n, hq, hk, d, io, size, sign, i, scale)
            o, lse = m3attn.m3_attention(*(x.to(DEV).unsqueeze(0) for x in (q, k, v)), scale=scale, save_lse=True)
            torch.cuda.synchronize()
            seen = torch.ones(n, n, dtype=torch.bool).tril()
            for h in sorted({0, hq // 2, hq - 1}):
                j = h // (hq // hk)
                want, tol, wl, tl = attend(q[:, h], k[:, j], v[:, j], scale, seen, io)
                assert_close(o[0, :, h], want, tol, "o %g %g" % (size, scale))
                assert_close(lse[0, h], wl, tl, "lse %g %g" % (size, scale))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("hq,hk,d,page,lens", [(4, 2, 64, 32, [1, 40, 700]), (3, 1, 128, 64, [5000, 130]),
                                               (20, 1, 128, 7, [300, 3000])])
def test_token_scores_far_from_zero(io, sign, hq, hk, d, page, lens):
    """One piece and several, of scores that the first pieces have alone or not."""
    io = IO[io]
    need = [-(-n // page) for n in lens]
    g = torch.Generator().manual_seed(1)
    order, table, at = torch.randperm(sum(need), generator=g), torch.full((len(lens), max(need)), -1, dtype=torch.int32), 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    for i, size in enumerate(SIZES):
        kc, vc = (torch.zeros(sum(need), hk, page, d, dtype=io) for _ in range(2))
        rows = []
        for s, n in enumerate(lens):
            q, k, v = exact_inputs(n, hq, hk, d, io, size, sign, 10 * i + s, 1.0)
            pos = torch.arange(n)
            kc[table[s, pos // page].long(), :, pos % page] = k
            vc[table[s, pos // page].long(), :, pos % page] = v
            rows.append((q[0], k, v))
        lse = torch.empty(len(lens), hq, device=DEV)
        o = m3attn.m3_attention_step(torch.stack([r[0] for r in rows]).to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV),
                                     torch.tensor(lens, dtype=torch.int32).to(DEV), scale=1.0, lse=lse)
        torch.cuda.synchronize()
        for s, (q, k, v) in enumerate(rows):
            for h in (0, hq - 1):
                j = h // (hq // hk)
                want, tol, wl, tl = attend(q[h:h + 1], k[:, j], v[:, j], 1.0, torch.ones(1, lens[s], dtype=torch.bool), io)
                assert_close(o[s, h], want[0], tol[0], "o %g" % size)
                assert_close(lse[s, h:h + 1], wl, tl, "lse %g" % size)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_token_scores_of_minus_infinity(io):
    """Positions that all score -inf are 0 / 0, as a prompt's row is; positions that are not there give zeros."""
    io, d, page, hq = IO[io], 64, 16, 4
    g = torch.Generator().manual_seed(3)
    kc, vc = (torch.randn(40, 1, page, d, generator=g).to(io) for _ in range(2))
    q = torch.randn(5, hq, d, generator=g).to(io)
    kc[:, 0, :, 0] = 0.0
    q[:, :, 0] = 1.0
    kc[:36, 0, :, 0] = float("-inf")
    table = torch.stack([torch.arange(36, dtype=torch.int32)] * 5)
    table[1, :] = -1
    table[2, 2] = 38                      # one page of other scores
    table[3, :20] = 50                    # no pages, then -inf
    lens = torch.tensor([36 * page, 36 * page, 36 * page, 36 * page, 3], dtype=torch.int32)
    lse = torch.empty(5, hq, device=DEV)
    o = m3attn.m3_attention_step(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), lens.to(DEV), lse=lse)
    short = m3attn.m3_attention_step(q.to(DEV), kc.to(DEV), vc.to(DEV), table[:, :1].contiguous().to(DEV), lens.to(DEV))
    torch.cuda.synchronize()
    for s in (0, 3, 4):
        assert torch.isnan(o[s].float()).all() and (lse[s] == float("-inf")).all(), s
    assert (o[1] == 0).all() and (lse[1] == float("-inf")).all()
    assert torch.isnan(short[[0, 2, 4]].float()).all() and (short[[1, 3]] == 0).all()
    k, v = kc[38, 0].double(), vc[38, 0].double()
    for h in range(hq):
        p = torch.softmax(k @ q[2, h].double() / 8, 0)
        e = (d + 24) * U32 * 8 + half_step(io)    # of scores below 8
        assert_close(o[2, h], p @ v, e * (p @ v.abs() + (p @ v).abs()), "o")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [2.0 ** -149, 1e-41, 1e-38, 1e-30, 2.3e38])
@pytest.mark.parametrize("h", [2, 130])
def test_scales_at_the_ends_of_the_range(io, scale, h):
    """All scores all but equal: means of the values."""
    io, n, d, page = IO[io], 290, 64, 16
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(1, n, h, d, generator=g).to(io) for _ in range(3))
    if scale > 1:
        q.zero_()
    o, lse = m3attn.m3_attention(q.to(DEV), k.to(DEV), v.to(DEV), scale=scale, save_lse=True)
    pages = -(-n // page)
    kc, vc = (torch.zeros(pages, h, page, d, dtype=io, device=DEV) for _ in range(2))
    table = torch.arange(pages, dtype=torch.int32, device=DEV).unsqueeze(0)
    m3attn.m3_cache_append(k.to(DEV), v.to(DEV), kc, vc, table)
    o1 = m3attn.m3_attention_step(q[:, -1].contiguous().to(DEV), kc, vc, table, torch.tensor([n], dtype=torch.int32, device=DEV),
                                  scale=scale)
    torch.cuda.synchronize()
    count = torch.arange(1, n + 1).double().view(n, 1, 1)
    want, size = v[0].double().cumsum(0) / count, v[0].double().abs().cumsum(0) / count
    # scores of up to 2^-90 are nothing beside 1; a probability and the sum are off by 16 units and one per addition
    tol = (2 * (16 + n) * U32 + (half_step(io) if io is torch.bfloat16 else 0.0)) * size
    assert_close(o[0], want, tol, "o")
    assert_close(o1[0], want[-1], tol[-1], "token")
    want = count.view(n).log().expand(h, n)
    assert_close(lse[0], want, (32 + n + 8 * want) * U32, "lse")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("h", [2, 130])
def test_scores_at_the_ends_of_the_range(io, sign, h):
    """Scores whose products with log2 e are beyond fp32."""
    io, n, d, page = IO[io], 200, 64, 16
    g = torch.Generator().manual_seed(5)
    q, k = torch.zeros(n, h, d), torch.zeros(n, h, d)
    q[:, :, 9], k[:, :, 9] = 2.0 ** 60, torch.where(torch.rand(n, h, generator=g) < 0.5, 1.75, 1.5) * sign * 2.0 ** 67
    if sign < 0:
        k[:70] = k[:70].clamp(max=0).where(k[:70] != -1.5 * 2.0 ** 67, torch.tensor(-1.75 * 2.0 ** 67))
    v = torch.randn(n, h, d, generator=g)
    q, k, v = q.to(io), k.to(io), v.to(io)
    o, lse = m3attn.m3_attention(*(x.to(DEV).unsqueeze(0) for x in (q, k, v)), scale=1.0, save_lse=True)
    pages = -(-n // page)
    kc, vc = (torch.zeros(pages, h, page, d, dtype=io, device=DEV) for _ in range(2))
    table = torch.arange(pages, dtype=torch.int32, device=DEV).unsqueeze(0)
    m3attn.m3_cache_append(k.to(DEV).unsqueeze(0), v.to(DEV).unsqueeze(0), kc, vc, table)
    lse1 = torch.empty(1, h, device=DEV)
    o1 = m3attn.m3_attention_step(q[-1:].to(DEV), kc, vc, table, torch.tensor([n], dtype=torch.int32, device=DEV), scale=1.0,
                                  lse=lse1)
    torch.cuda.synchronize()
    seen = torch.ones(n, n, dtype=torch.bool).tril()
    for i in (0, h - 1):
        want, tol, wl, tl = attend(q[:, i], k[:, i], v[:, i], 1.0, seen, io)
        assert_close(o[0, :, i], want, tol, "o")
        assert_close(lse[0, i], wl, tl, "lse")
        assert_close(o1[0, i], want[-1], tol[-1], "token")
        assert_close(lse1[0, i], wl[-1], tl[-1], "token's lse")
