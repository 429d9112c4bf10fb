"""The attention operators in a row, as an attention layer of a hybrid stack uses them: prompts in training (rotation,
attention, both backward), prompts of different lengths in serving (rotation and cache in one call, attention), and
tokens decoded one by one behind them, each checked against the formulas in 64 bits; and beside the other operators
of a block (norm, clipping)."""
from __future__ import annotations

import pytest
import torch

import attn_ref
from block_ref import U32, assert_close, half_step
from state_space_sequence_m3_amd import m3attn, m3block

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def frequencies(r):
    return (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prompt_then_tokens(io):
    """Prefill into the cache, then decode: every token's output is that of causal attention over its whole sequence, from
    what the calls themselves put into the cache."""
    io = IO[io]
    hq, hk, d, page, steps = 8, 2, 64, 16, 4
    lens = [37, 0, 150, 1]
    b, t = len(lens), sum(lens)
    g = torch.Generator().manual_seed(1)
    new = lambda *s: torch.randn(*s, generator=g).to(io)
    freq = frequencies(d)
    total = [n + steps for n in lens]
    need = [-(-n // page) for n in total]
    order, table, at = torch.randperm(sum(need), generator=g), torch.full((b, max(need)), -1, dtype=torch.int32), 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    kc, vc = (torch.zeros(sum(need), hk, page, d, dtype=io, device=DEV) for _ in range(2))
    td, fd = table.to(DEV), freq.to(DEV)
    q, k, v = new(t, hq, d), new(t, hk, d), new(t, hk, d)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    length = torch.tensor(lens, dtype=torch.int32).to(DEV)
    qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    qr = m3attn.m3_cache_append(kd, vd, kc, vc, td, length, q=qd, inv_freq=fd, cu_seqlens=cu, q_out=qd, k_out=kd)
    o = m3attn.m3_attention(qr, kd, vd, cu)
    torch.cuda.synchronize()
    assert qr is qd
    pos = torch.cat([torch.arange(n) for n in lens])
    want, tol = attn_ref.rotate(k, pos, freq, False)
    assert_close(kd, want, tol, "rotated k")
    ref = attn_ref.prompt(qd.cpu(), kd.cpu(), v, lens)
    assert_close(o, ref["o"], ref["tol"]["o"], "prompt")
    for step in range(steps):
        q1, k1, v1 = new(b, 1, hq, d), new(b, 1, hk, d), new(b, 1, hk, d)
        length += 1
        qr = m3attn.m3_cache_append(k1.to(DEV), v1.to(DEV), kc, vc, td, length, q=q1.to(DEV), inv_freq=fd)
        o = m3attn.m3_attention_step(qr[:, 0], kc, vc, td, length)
        torch.cuda.synchronize()
        at = torch.tensor(lens) + step
        want, tol = attn_ref.rotate(q1[:, 0], at, freq, False)
        assert_close(qr[:, 0], want, tol, "rotated q")
        kh, vh = kc.cpu(), vc.cpu()
        keys, values = [], []
        for s in range(b):
            n = lens[s] + step + 1
            ids = table[s, :-(-n // page)].long()
            keys.append(kh[ids].transpose(0, 1).flatten(1, 2)[:, :n])
            values.append(vh[ids].transpose(0, 1).flatten(1, 2)[:, :n])
            assert torch.equal(values[-1][:, -1], v1[s, 0])
            want, tol = attn_ref.rotate(k1[s], at[s:s + 1], freq, False)
            assert_close(keys[-1][:, -1], want[0], tol[0], "cached k")
        ref = attn_ref.step(qr[:, 0].cpu(), keys, values)
        assert_close(o, ref["o"], ref["tol"]["o"], "token")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_is_the_last_row_of_the_prompt(io):
    """The two kernels agree with each other, within what each may be off from the formula."""
    io = IO[io]
    n, hq, hk, d, page = 700, 4, 2, 128, 32
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(1, n, h, d, generator=g).to(io).to(DEV) for h in (hq, hk, hk))
    pages = -(-n // page)
    kc, vc = (torch.zeros(pages, hk, page, d, dtype=io, device=DEV) for _ in range(2))
    table = torch.arange(pages, dtype=torch.int32, device=DEV).flip(0).unsqueeze(0).contiguous()
    m3attn.m3_cache_append(k, v, kc, vc, table)
    o, lse = m3attn.m3_attention(q, k, v, save_lse=True)
    lse1 = torch.empty(1, hq, device=DEV)
    o1 = m3attn.m3_attention_step(q[:, -1], kc, vc, table, torch.tensor([n], dtype=torch.int32, device=DEV), lse=lse1)
    torch.cuda.synchronize()
    ref = attn_ref.prompt(q[0].cpu(), k[0].cpu(), v[0].cpu(), [n])
    for got in (o[0, -1], o1[0]):
        assert_close(got, ref["o"][-1], ref["tol"]["o"][-1], "o")
    for got in (lse[0, :, -1], lse1[0]):
        assert_close(got, ref["lse"][:, -1], ref["tol"]["lse"][:, -1], "lse")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_training_step_of_a_layer(io):
    """Norm, projections, rotation, attention, and all of it backwards to the projections' weights, with clipping: the
    gradients are those that torch's autograd finds for the formulas in 64 bits, within 2 % (fp32: 2e-5) of their norm."""
    dt = IO[io]
    b, n, hq, hk, d = 2, 160, 4, 2, 64
    width = hq * d
    g = torch.Generator().manual_seed(3)
    x = torch.randn(b, n, width, generator=g).to(dt)
    w = torch.randn(width, (hq + 2 * hk) * d, generator=g) / width ** 0.5
    wo = torch.randn(width, width, generator=g) / width ** 0.5
    dy = torch.randn(b, n, width, generator=g).to(dt)
    freq = frequencies(d)

    # 64 bits
    x64, w64, wo64 = (t.double().requires_grad_() for t in (x, w.to(dt), wo.to(dt)))
    r = x64 / torch.sqrt(x64.square().mean(-1, keepdim=True) + 1e-5)
    p = (r @ w64).unflatten(-1, (hq + 2 * hk, d))
    ang = torch.outer(torch.arange(n).double(), freq.double())
    cos, sin = ang.cos()[None, :, None], ang.sin()[None, :, None]
    turn = lambda t: torch.stack([t[..., ::2] * cos - t[..., 1::2] * sin, t[..., ::2] * sin + t[..., 1::2] * cos], -1).flatten(-2)
    q, k, v = turn(p[:, :, :hq]), turn(p[:, :, hq:hq + hk]), p[:, :, hq + hk:]
    s = torch.einsum("bihd,bjhd->bhij", q, k.repeat_interleave(hq // hk, 2)) * d ** -0.5
    s = s.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), float("-inf"))
    o = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v.repeat_interleave(hq // hk, 2))
    (o.flatten(2) @ wo64).backward(dy.double())

    # the operators, slices of one projection throughout, gradients into slices of one buffer
    xd, wd, wod, dyd, fd = x.to(DEV), w.to(dt).to(DEV), wo.to(dt).to(DEV), dy.to(DEV), freq.to(DEV)
    r, _, _, _ = m3block.m3_rmsnorm(xd)
    p = (r.view(-1, width) @ wd).view(b, n, hq + 2 * hk, d)
    q, k, v = p[:, :, :hq], p[:, :, hq:hq + hk], p[:, :, hq + hk:]
    m3attn.m3_cache_append(k, None, q=q, inv_freq=fd, q_out=q, k_out=k)
    o, lse = m3attn.m3_attention(q, k, v, save_lse=True)
    do = (dyd.view(-1, width) @ wod.t().contiguous()).view(b, n, hq, d)
    dp = torch.empty_like(p)
    grads = {"q": dp[:, :, :hq], "k": dp[:, :, hq:hq + hk], "v": dp[:, :, hq + hk:]}
    m3attn.m3_attention_backward(q, k, v, o, lse, do, grads=grads)
    m3attn.m3_cache_append(grads["k"], None, q=grads["q"], inv_freq=-fd, q_out=grads["q"], k_out=grads["k"])
    dw = r.view(-1, width).t().contiguous() @ dp.view(b * n, -1)
    dwo = o.view(-1, width).t().contiguous() @ dyd.view(-1, width)
    dr = (dp.view(b * n, -1) @ wd.t().contiguous()).view(b, n, width)
    dx, _ = m3block.m3_rmsnorm_backward(xd, dr)
    clipped, stats = m3block.m3_grad_clip([dw, dwo], 1.0, out=[torch.empty_like(dw), torch.empty_like(dwo)])
    torch.cuda.synchronize()
    # about ten roundings to bf16 on the way, each 2^-8 at most and some 2^-9 as norms; fp32: sums of up to 512 products
    tol = 10 * half_step(torch.bfloat16) / 2 if io == "bf16" else 512 * U32 / 2
    for name, got, want in (("dw", dw, w64.grad), ("dwo", dwo, wo64.grad), ("dx", dx, x64.grad)):
        off = float((got.cpu().double() - want).norm() / want.norm())
        assert off <= tol, (name, off, tol)
    norm = float(torch.sqrt(dw.double().square().sum() + dwo.double().square().sum()))
    assert abs(float(stats[0]) - norm) <= 1e-5 * norm
    assert abs(float(torch.stack([c.double().square().sum() for c in clipped]).sum().sqrt()) - 1.0) <= 1e-2


def test_two_graphs_at_once():
    """Two captured decoding steps with caches and workspaces of their own, replayed at the same time."""
    b, hq, hk, d, page, n = 4, 8, 2, 128, 64, 1000
    g = torch.Generator().manual_seed(4)
    pages = -(-n // page)
    sets = []
    for _ in range(2):
        kc, vc = (torch.randn(b * pages, hk, page, d, generator=g).bfloat16().to(DEV) for _ in range(2))
        table = torch.randperm(b * pages, generator=g).view(b, pages).to(torch.int32).to(DEV)
        lens = torch.randint(1, n, (b,), generator=g).to(torch.int32).to(DEV)
        q = torch.randn(b, hq, d, generator=g).bfloat16().to(DEV)
        sets.append((q, kc, vc, table, lens))
    want = [m3attn.m3_attention_step(*s) for s in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(m3attn.m3_attention_step(*s))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
