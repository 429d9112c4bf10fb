"""m3_attention and its backward pass against the formulas in 64 bits: both types, every width class of heads, groups,
lengths around the kernels' blocks of 32, 64 and 128 tokens, packed batches with empty sequences, strides of
projections and of heads before tokens, infinities and NaN in later tokens.  Bounds: tests/attn_ref.py."""
from __future__ import annotations

import pytest
import torch

import attn_ref
from block_ref import assert_close
from state_space_sequence_m3_amd import m3attn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def draw(t, hq, hk, d, io, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda h: torch.randn(t, h, d, generator=g).to(io)
    return r(hq), r(hk), r(hk), r(hq)


def offsets(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)


def assert_lse(lse, ref):
    assert_close(lse, ref["lse"], ref["tol"]["lse"], "lse")


def check_packed(q, k, v, dout, lens, scale=None):
    ref = attn_ref.prompt(q, k, v, lens, scale, dout)
    qd, kd, vd, dd, cu = q.to(DEV), k.to(DEV), v.to(DEV), dout.to(DEV), offsets(lens)
    o, lse = m3attn.m3_attention(qd, kd, vd, cu, scale, save_lse=True)
    g = m3attn.m3_attention_backward(qd, kd, vd, o, lse, dd, cu, scale)
    torch.cuda.synchronize()
    n = sum(lens)
    assert_close(o[:n], ref["o"][:n], ref["tol"]["o"][:n], "o")
    assert_close(lse[:, :n], ref["lse"][:, :n], ref["tol"]["lse"][:, :n], "lse")
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        assert_close(g[key][:n], ref[name][:n], ref["tol"][name][:n], name)
    return o, lse, g


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 200, 257])
def test_lengths(io, n):
    """Dense batches of every remainder of the blocks."""
    b, hq, hk, d = 2, 4, 2, 64
    q, k, v, dout = draw(b * n, hq, hk, d, IO[io], n)
    ref = attn_ref.prompt(q, k, v, [n] * b, None, dout)
    qd, kd, vd, dd = (x.to(DEV).unflatten(0, (b, n)) for x in (q, k, v, dout))
    o, lse = m3attn.m3_attention(qd, kd, vd, save_lse=True)
    g = m3attn.m3_attention_backward(qd, kd, vd, o, lse, dd)
    torch.cuda.synchronize()
    assert_close(o.flatten(0, 1), ref["o"], ref["tol"]["o"], "o")
    assert_close(lse.transpose(0, 1).flatten(1), ref["lse"], ref["tol"]["lse"], "lse")
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        assert_close(g[key].flatten(0, 1), ref[name], ref["tol"][name], name)
    assert torch.equal(o, m3attn.m3_attention(qd, kd, vd))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [8, 16, 24, 32, 40, 64, 72, 80, 96, 104, 112, 120, 128])
def test_head_widths(io, d):
    lens = [70, 0, 1, 145]
    q, k, v, dout = draw(sum(lens), 2, 1, d, IO[io], d)
    check_packed(q, k, v, dout, lens)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (8, 1), (6, 2), (5, 5), (16, 8), (24, 8)])
def test_groups(io, hq, hk):
    lens = [97, 40]
    q, k, v, dout = draw(sum(lens), hq, hk, 128, IO[io], hq * 100 + hk)
    check_packed(q, k, v, dout, lens)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_longer(io):
    lens = [1100, 130, 0, 515]
    q, k, v, dout = draw(sum(lens), 2, 1, 128, IO[io], 3)
    check_packed(q, k, v, dout, lens)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_many_sequences(io):
    """More sequences than lanes, empty ones at both ends and in a row; rows past the last are left as they were."""
    g = torch.Generator().manual_seed(9)
    lens = [0, 0] + torch.randint(0, 9, (150,), generator=g).tolist() + [0] * 70 + [130, 3, 0]
    n, more = sum(lens), 37
    q, k, v, dout = draw(n + more, 2, 2, 32, IO[io], 5)
    ref = attn_ref.prompt(q[:n], k[:n], v[:n], lens, None, dout[:n])
    qd, kd, vd, dd, cu = q.to(DEV), k.to(DEV), v.to(DEV), dout.to(DEV), offsets(lens)
    o = torch.full_like(qd, 7.0)
    lse = torch.full((2, n + more), 7.0, device=DEV)
    m3attn.m3_attention(qd, kd, vd, cu, o=o, lse=lse)
    grads = {x: torch.full_like(t, 7.0) for x, t in (("q", qd), ("k", kd), ("v", vd))}
    m3attn.m3_attention_backward(qd, kd, vd, o, lse, dd, cu, grads=grads)
    torch.cuda.synchronize()
    assert_close(o[:n], ref["o"], ref["tol"]["o"], "o")
    assert_close(lse[:, :n], ref["lse"], ref["tol"]["lse"], "lse")
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        assert_close(grads[key][:n], ref[name], ref["tol"][name], name)
    for t in (o[n:], lse[:, n:], grads["q"][n:], grads["k"][n:], grads["v"][n:]):
        assert (t == 7.0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_no_tokens(io):
    x = torch.empty(0, 2, 64, dtype=IO[io], device=DEV)
    o, lse = m3attn.m3_attention(x, x, x, offsets([0, 0]), save_lse=True)
    g = m3attn.m3_attention_backward(x, x, x, o, lse, x, offsets([0, 0]))
    assert o.shape == x.shape and lse.shape == (2, 0) and g["k"].shape == x.shape
    x = torch.full((3, 2, 64), 7.0, dtype=IO[io], device=DEV)   # tokens, but no sequence has any
    o = torch.full_like(x, 7.0)
    m3attn.m3_attention(x, x, x, offsets([]), o=o)
    m3attn.m3_attention(x, x, x, offsets([0, 0]), o=o)
    torch.cuda.synchronize()
    assert (o == 7.0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["projection", "heads first", "stacked"])
def test_strides(io, layout):
    """Inputs and gradients as slices of one projection, as [b, H, L, D], and as [b, 3, H, L, D]."""
    b, n, h, d = 2, 150, 2, 64
    q, k, v, dout = draw(b * n, h, h, d, IO[io], 11)
    ref = attn_ref.prompt(q, k, v, [n] * b, None, dout)

    def buffers():
        if layout == "projection":
            wide = torch.full((b, n, 3 * h + 1, d), 5.0, dtype=IO[io], device=DEV)
            return wide, [wide[:, :, i * h:(i + 1) * h] for i in range(3)]
        if layout == "heads first":
            wide = [torch.empty(b, h, n, d, dtype=IO[io], device=DEV) for _ in range(3)]
            return None, [t.transpose(1, 2) for t in wide]
        wide = torch.empty(b, 3, h, n, d, dtype=IO[io], device=DEV)
        return None, [wide[:, i].transpose(1, 2) for i in range(3)]

    _, ins = buffers()
    wide, outs = buffers()
    for t, x in zip(ins, (q, k, v)):
        t.copy_(x.unflatten(0, (b, n)))
    dd = dout.to(DEV).unflatten(0, (b, n)).transpose(1, 2).contiguous().transpose(1, 2)
    o = torch.empty(b, h, n, d, dtype=IO[io], device=DEV).transpose(1, 2)
    o, lse = m3attn.m3_attention(*ins, o=o, save_lse=True)
    g = m3attn.m3_attention_backward(*ins, o, lse, dd, grads=dict(zip("qkv", outs)))
    torch.cuda.synchronize()
    assert_close(o.flatten(0, 1), ref["o"], ref["tol"]["o"], "o")
    for name, key, t in (("dq", "q", outs[0]), ("dk", "k", outs[1]), ("dv", "v", outs[2])):
        assert g[key] is t
        assert_close(t.flatten(0, 1), ref[name], ref["tol"][name], name)
    if wide is not None:
        assert (wide[:, :, 3 * h:] == 5.0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_shared_keys_as_a_stride_of_zero(io):
    """One key head, given as four by a stride of 0."""
    lens = [90, 33]
    q, k, v, _ = draw(sum(lens), 4, 1, 64, IO[io], 12)
    ref = attn_ref.prompt(q, k, v, lens)
    kd, vd = k.to(DEV), v.to(DEV)
    o = m3attn.m3_attention(q.to(DEV), kd.expand(-1, 4, -1), vd.expand(-1, 4, -1), offsets(lens))
    torch.cuda.synchronize()
    assert_close(o, ref["o"], ref["tol"]["o"], "o")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.01, 0.5, 3.0])
def test_scales(io, scale):
    """Flat and very peaked rows."""
    lens = [140]
    q, k, v, dout = draw(sum(lens), 2, 1, 64, IO[io], 13)
    check_packed(q, k, v, dout, lens, scale)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_growing_scores(io):
    """Scores that grow along the keys move the running maximum in every block."""
    n, d = 300, 64
    q, k, v, dout = draw(n, 1, 1, d, IO[io], 14)
    k = (k.float() * 0.1 + torch.arange(n).view(n, 1, 1) / n * q.float().mean(0, keepdim=True).sign() * 3).to(IO[io])
    q = (q.float() * 0.1 + q.float().mean(0, keepdim=True).sign() * 2).to(IO[io])
    check_packed(q, k, v, dout, [n])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("where", ["k", "v"])
def test_later_tokens_do_not_reach_a_row(io, bad, where):
    """A key or value that is not finite leaves all rows before it, and the other sequence, as they are."""
    lens, d = [150, 20], 64
    q, k, v, _ = draw(sum(lens), 2, 1, d, IO[io], 15)
    cu = offsets(lens)
    want = m3attn.m3_attention(q.to(DEV), k.to(DEV), v.to(DEV), cu)
    for at in (0, 5, 31, 70, 127, 149):
        x = {"k": k.clone(), "v": v.clone()}
        x[where][at, 0, 3] = bad
        o, lse = m3attn.m3_attention(q.to(DEV), x["k"].to(DEV), x["v"].to(DEV), cu, save_lse=True)
        torch.cuda.synchronize()
        tol = 2.0 ** -6 if io == "bf16" else 2.0 ** -18   # the block is added up in another order, unrounded
        assert torch.allclose(o[:at].float(), want[:at].float(), atol=tol, rtol=tol), at
        assert torch.equal(o[150:], want[150:])
        if where == "v":
            assert torch.isfinite(lse).all()
            touched = o[at:150, :, 3].float()
            assert (torch.isnan(touched) if bad != bad else touched == bad).all(), at
            rest = torch.cat([o[at:150, :, :3], o[at:150, :, 4:]], 2)
            assert torch.isfinite(rest.float()).all()
        elif bad != bad:
            assert torch.isnan(o[at:150].float()).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_scores_of_minus_infinity(io):
    """A row whose first keys score -inf takes the others alone; one with nothing else is NaN, as 0 / 0 is."""
    n, d = 70, 64
    q, k, v, _ = draw(n, 1, 1, d, IO[io], 16)
    q[:, 0, 0], k[:, 0, 0] = 1.0, 0.0
    k[:40, 0, 0] = float("-inf")
    o = m3attn.m3_attention(q.to(DEV), k.to(DEV), v.to(DEV), offsets([n]))
    seen = torch.ones(n, n, dtype=torch.bool).tril()
    seen[:, :40] = False
    k[:40, 0, 0] = 0.0
    a = attn_ref.attend(q[:, 0].double(), k[:, 0].double(), v[:, 0].double(), d ** -0.5, seen, IO[io])
    torch.cuda.synchronize()
    assert torch.isnan(o[:40].float()).all()
    assert_close(o[40:, 0], a["o"][40:], a["tol"]["o"][40:], "o")


def test_gradient_against_differences():
    """fp32 gradients along random directions against central differences of the 64-bit formula."""
    lens, d = [40, 7, 66], 32
    q, k, v, dout = draw(sum(lens), 4, 2, d, torch.float32, 17)
    cu = offsets(lens)
    o, lse = m3attn.m3_attention(q.to(DEV), k.to(DEV), v.to(DEV), cu, save_lse=True)
    g = m3attn.m3_attention_backward(q.to(DEV), k.to(DEV), v.to(DEV), o, lse, dout.to(DEV), cu)
    gen = torch.Generator().manual_seed(18)
    ref = attn_ref.prompt(q, k, v, lens, None, dout)
    for name, key, x in (("dq", "q", q), ("dk", "k", k), ("dv", "v", v)):
        way = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        eps = 1e-5
        vals = []
        for sign in (1, -1):
            y = {"q": q.double(), "k": k.double(), "v": v.double()}
            y[key] = y[key] + sign * eps * way
            vals.append(float((attn_ref.prompt(y["q"], y["k"], y["v"], lens)["o"] * dout.double()).sum()))
        diff = (vals[0] - vals[1]) / (2 * eps)
        got = float((g[key].cpu().double() * way).sum())
        # eps^2 of the third derivative, fp64's own rounding over eps, and the gradient's bound
        bound = float(((ref["tol"][name] + 2.0 ** -24 * ref[name].abs()) * way.abs()).sum()) + 1e-6 * (1 + abs(diff))
        assert abs(got - diff) <= bound, (name, got, diff, bound)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_streams_and_repeats(io):
    """On a stream of its own, twice: equal bits."""
    lens = [300, 44]
    q, k, v, dout = (x.to(DEV) for x in draw(sum(lens), 4, 2, 64, IO[io], 19))
    cu = offsets(lens)
    o, lse = m3attn.m3_attention(q, k, v, cu, save_lse=True)
    g = m3attn.m3_attention_backward(q, k, v, o, lse, dout, cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        o2, lse2 = m3attn.m3_attention(q, k, v, cu, save_lse=True, stream=s)
        g2 = m3attn.m3_attention_backward(q, k, v, o2, lse2, dout, cu, stream=s)
        s.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert all(torch.equal(g[x], g2[x]) for x in "qkv")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_graph(io):
    """A captured training step, replayed with new inputs between eager work."""
    b, n, hq, hk, d = 2, 150, 4, 2, 64
    q, k, v, dout = (x.to(DEV).unflatten(0, (b, n)) for x in draw(b * n, hq, hk, d, IO[io], 20))

    def once():
        o, lse = m3attn.m3_attention(q, k, v, save_lse=True)
        return o, m3attn.m3_attention_backward(q, k, v, o, lse, dout)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, g = once()
    for i in range(4):
        for t, x in zip((q, k, v, dout), draw(b * n, hq, hk, d, IO[io], 30 + i)):
            t.copy_(x.unflatten(0, (b, n)))
        want_o, want = once()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want_o)
        assert all(torch.equal(g[x], want[x]) for x in "qkv")


# Batches above are small, so blocks of 32 rows whose waves share the other axis; with many heads the kernels take
# blocks of 128 rows.  What the heads' number decides: rows (over 256 blocks), keys (over 256, fp32 512), and into how
# many parts the heads of a group are split for dk and dv (up to 1024 blocks; small ones up to 128).

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 40, 64, 96, 104, 128])
def test_many_heads(io, d):
    lens = [129, 0, 1, 300, 33, 64]
    q, k, v, dout = draw(sum(lens), 180, 180, d, IO[io], 40 + d)
    check_packed(q, k, v, dout, lens)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n", [100, 128, 256, 290])
def test_many_heads_dense(io, n):
    b, hq, hk, d = 2, 320, 160, 64
    q, k, v, dout = draw(b * n, hq, hk, d, IO[io], n)
    ref = attn_ref.prompt(q, k, v, [n] * b, None, dout)
    qd, kd, vd, dd = (x.to(DEV).unflatten(0, (b, n)) for x in (q, k, v, dout))
    o, lse = m3attn.m3_attention(qd, kd, vd, save_lse=True)
    g = m3attn.m3_attention_backward(qd, kd, vd, o, lse, dd)
    torch.cuda.synchronize()
    assert_close(o.flatten(0, 1), ref["o"], ref["tol"]["o"], "o")
    assert_close(lse.transpose(0, 1).flatten(1), ref["lse"], ref["tol"]["lse"], "lse")
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        assert_close(g[key].flatten(0, 1), ref[name], ref["tol"][name], name)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk,d", [(160, 40, 64), (240, 40, 128), (96, 16, 32), (30, 5, 96), (12, 2, 128)])
def test_groups_split_over_workgroups(io, hq, hk, d):
    """dk and dv out of parts, dense and packed with rows behind the last sequence."""
    lens, more = [200, 0, 33], 9
    n = sum(lens)
    q, k, v, dout = draw(n + more, hq, hk, d, IO[io], hq + d)
    ref = attn_ref.prompt(q[:n], k[:n], v[:n], lens, None, dout[:n])
    qd, kd, vd, dd, cu = q.to(DEV), k.to(DEV), v.to(DEV), dout.to(DEV), offsets(lens)
    o, lse = m3attn.m3_attention(qd, kd, vd, cu, save_lse=True)
    wide = torch.full((n + more, hq + 2 * hk, d), 7.0, dtype=IO[io], device=DEV)
    grads = {"q": wide[:, :hq], "k": wide[:, hq:hq + hk], "v": wide[:, hq + hk:]}
    m3attn.m3_attention_backward(qd, kd, vd, o, lse, dd, cu, grads=grads)
    torch.cuda.synchronize()
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        assert_close(grads[key][:n], ref[name], ref["tol"][name], name)
    assert (wide[n:] == 7.0).all()
    b, rows = 2, 116
    x = [t[:b * rows].to(DEV).unflatten(0, (b, rows)) for t in (q, k, v, dout)]
    ref = attn_ref.prompt(q[:b * rows], k[:b * rows], v[:b * rows], [rows] * b, None, dout[:b * rows])
    o, lse = m3attn.m3_attention(*x[:3], save_lse=True)
    first = [torch.empty(b, h, rows, d, dtype=IO[io], device=DEV).transpose(1, 2) for h in (hq, hk, hk)]
    g = m3attn.m3_attention_backward(*x[:3], o, lse, x[3], grads=dict(zip("qkv", first)))
    torch.cuda.synchronize()
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        assert_close(g[key].flatten(0, 1), ref[name], ref["tol"][name], name)


@pytest.mark.parametrize("hq,hk,d,lens", [(36, 36, 128, [1100]), (40, 40, 72, [1500, 600, 1024]), (24, 12, 128, [1024, 1290]),
                                          (33, 33, 96, [1025])])
def test_long_sequences_of_many_heads(hq, hk, d, lens):
    """dk and dv by workgroups of 256 keys."""
    q, k, v, dout = draw(sum(lens), hq, hk, d, torch.bfloat16, d)
    if len(lens) > 1:
        check_packed(q, k, v, dout, lens)
        return
    ref = attn_ref.prompt(q, k, v, lens, None, dout)
    x = [t.to(DEV).unsqueeze(0) for t in (q, k, v, dout)]
    o, lse = m3attn.m3_attention(*x[:3], save_lse=True)
    g = m3attn.m3_attention_backward(*x[:3], o, lse, x[3])
    torch.cuda.synchronize()
    assert_close(o[0], ref["o"], ref["tol"]["o"], "o")
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        assert_close(g[key][0], ref[name], ref["tol"][name], name)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_later_tokens_do_not_reach_a_row_of_many_heads(io, bad):
    lens, d, h = [300, 20], 64, 130
    q, k, v, _ = draw(sum(lens), h, 1, d, IO[io], 41)
    cu = offsets(lens)
    want = m3attn.m3_attention(q.to(DEV), k.to(DEV), v.to(DEV), cu)
    for at in (0, 40, 127, 200, 299):
        x = v.clone()
        x[at, 0, 3] = bad
        o = m3attn.m3_attention(q.to(DEV), k.to(DEV), x.to(DEV), cu)
        torch.cuda.synchronize()
        tol = 2.0 ** -6 if io == "bf16" else 2.0 ** -18
        assert torch.allclose(o[:at].float(), want[:at].float(), atol=tol, rtol=tol), at
        assert torch.equal(o[300:], want[300:])
        touched = o[at:300, :, 3].float()
        assert (torch.isnan(touched) if bad != bad else touched == bad).all(), at


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_graph_of_many_heads(io):
    """Blocks of 128 rows and split groups, captured and replayed between eager work: equal bits."""
    b, n, hq, hk, d = 2, 150, 160, 40, 128
    q, k, v, dout = (x.to(DEV).unflatten(0, (b, n)) for x in draw(b * n, hq, hk, d, IO[io], 42))

    def once():
        o, lse = m3attn.m3_attention(q, k, v, save_lse=True)
        return o, m3attn.m3_attention_backward(q, k, v, o, lse, dout)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, g = once()
    for i in range(4):
        for t, x in zip((q, k, v, dout), draw(b * n, hq, hk, d, IO[io], 50 + i)):
            t.copy_(x.unflatten(0, (b, n)))
        want_o, want = once()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want_o)
        assert all(torch.equal(g[x], want[x]) for x in "qkv")


def test_tokens_far_apart():
    """Rows over 4 GB of a buffer: addresses beyond 32 bits."""
    n, d, token = 2100, 64, 1 << 20
    room = torch.empty(n * token, dtype=torch.bfloat16, device=DEV)
    rows = lambda at: room.as_strided((n, 1, d), (token, d, 1), at * d)
    q, k, v, dout = draw(n, 1, 1, d, torch.bfloat16, 43)
    ins = [rows(i) for i in range(4)]
    for t, x in zip(ins, (q, k, v, dout)):
        t.copy_(x)
    ref = attn_ref.prompt(q, k, v, [n], None, dout)
    cu = offsets([n])
    o, lse = m3attn.m3_attention(*ins[:3], cu, o=rows(4), save_lse=True)
    g = m3attn.m3_attention_backward(*ins[:3], o, lse, ins[3], cu, grads={x: rows(5 + i) for i, x in enumerate("qkv")})
    torch.cuda.synchronize()
    assert_close(o, ref["o"], ref["tol"]["o"], "o")
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        assert_close(g[key], ref[name], ref["tol"][name], name)


@pytest.mark.parametrize("io,hq,hk,d,lens", [("f32", 200, 40, 64, [116, 100]), ("f32", 71, 1, 32, [700]),
                                             ("bf16", 700, 100, 32, [300]), ("bf16", 350, 50, 72, [290, 0, 40, 350])])
def test_groups_split_into_uneven_parts(io, hq, hk, d, lens):
    """Groups of 5, 71 and 7 heads in fewer parts than heads, which no number of parts divides."""
    q, k, v, dout = draw(sum(lens), hq, hk, d, IO[io], hq)
    check_packed(q, k, v, dout, lens)
    if len(lens) > 1:
        return
    ref = attn_ref.prompt(q, k, v, lens, None, dout)
    x = [t.to(DEV).unsqueeze(0) for t in (q, k, v, dout)]
    o, lse = m3attn.m3_attention(*x[:3], save_lse=True)
    g = m3attn.m3_attention_backward(*x[:3], o, lse, x[3])
    torch.cuda.synchronize()
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        assert_close(g[key][0], ref[name], ref["tol"][name], name)


# Dense fp32 batches of many heads take two workgroups to a compute unit where heads have up to 96 elements, packed ones one.

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [8, 32, 40, 72, 96, 104, 128])
@pytest.mark.parametrize("n", [128, 290])
def test_many_heads_dense_widths(io, d, n):
    b, hq, hk = 2, 132, 132
    q, k, v, dout = draw(b * n, hq, hk, d, IO[io], n + d)
    ref = attn_ref.prompt(q, k, v, [n] * b, None, dout)
    qd, kd, vd, dd = (x.to(DEV).unflatten(0, (b, n)) for x in (q, k, v, dout))
    o, lse = m3attn.m3_attention(qd, kd, vd, save_lse=True)
    g = m3attn.m3_attention_backward(qd, kd, vd, o, lse, dd)
    torch.cuda.synchronize()
    assert_close(o.flatten(0, 1), ref["o"], ref["tol"]["o"], "o")
    assert_close(lse.transpose(0, 1).flatten(1), ref["lse"], ref["tol"]["lse"], "lse")
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        assert_close(g[key].flatten(0, 1), ref[name], ref["tol"][name], name)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("d", [32, 72, 96, 128])
def test_later_tokens_do_not_reach_a_row_of_dense_batches(io, bad, d):
    n, h = 300, 130
    q, k, v, _ = draw(n, h, 1, d, IO[io], 44)
    x = [t.to(DEV).unsqueeze(0) for t in (q, k, v)]
    want = m3attn.m3_attention(*x)[0]
    for at in (0, 40, 127, 200, 299):
        x[2] = v.clone().unsqueeze(0)
        x[2][0, at, 0, 3] = bad
        x[2] = x[2].to(DEV)
        o = m3attn.m3_attention(*x)[0]
        torch.cuda.synchronize()
        tol = 2.0 ** -6 if io == "bf16" else 2.0 ** -18   # the block is added up in another order, unrounded
        assert torch.allclose(o[:at].float(), want[:at].float(), atol=tol, rtol=tol), at
        touched = o[at:, :, 3].float()
        assert (torch.isnan(touched) if bad != bad else touched == bad).all(), at
        rest = torch.cat([o[at:, :, :3], o[at:, :, 4:]], 2)
        assert torch.isfinite(rest.float()).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gradients_of_broadcast_keys(io):
    """One key head given as four by a stride of 0: a gradient for each of the four."""
    lens = [90, 0, 33]
    q, k, v, dout = draw(sum(lens), 4, 1, 64, IO[io], 45)
    ref = attn_ref.prompt(q, k.repeat(1, 4, 1), v.repeat(1, 4, 1), lens, None, dout)
    kd, vd, cu = k.to(DEV).expand(-1, 4, -1), v.to(DEV).expand(-1, 4, -1), offsets(lens)
    o, lse = m3attn.m3_attention(q.to(DEV), kd, vd, cu, save_lse=True)
    g = m3attn.m3_attention_backward(q.to(DEV), kd, vd, o, lse, dout.to(DEV), cu)
    torch.cuda.synchronize()
    for name, key in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        assert_close(g[key], ref[name], ref["tol"][name], name)
