"""m3_cache_append and m3_attention_step against the formulas in 64 bits: both types, both pairings of the rotation,
page sizes that are powers of two and not, pages in any order and shared ones, empty sequences, lengths around the
pieces and tiles, head groups over 16, strides, numbers that are no page.  Bounds: tests/attn_ref.py."""
from __future__ import annotations

import pytest
import torch

import attn_ref
from block_ref import assert_close
from state_space_sequence_m3_amd import m3attn

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def frequencies(r):
    return (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / max(r, 1))).float()


def make_cache(totals, hk, page, d, io, seed, spare=3):
    """Caches with random contents, and a table of pages in no order."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in totals]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(totals), max(need + [0]) + 1), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    k, v = (torch.randn(pages, hk, page, d, generator=g).to(io) for _ in range(2))
    return k, v, table


def rows_of(cache, table, s, n):
    """[Hkv, n, D] of sequence s."""
    page = cache.shape[2]
    if n == 0:
        return cache.new_zeros(cache.shape[1], 0, cache.shape[3])
    ids = table[s, :-(-n // page)].long()
    return cache[ids].transpose(0, 1).flatten(1, 2)[:, :n]


def check_append(io, lens, pasts, hq, hk, d, page, rot, halves, packed, seed, with_q=True):
    io = IO[io]
    g = torch.Generator().manual_seed(seed)
    t, b = sum(lens), len(lens)
    q, k, v = (torch.randn(t, h, d, generator=g).to(io) for h in (hq, hk, hk))
    totals = [p + n for p, n in zip(pasts, lens)]
    kc, vc, table = make_cache(totals, hk, page, d, io, seed + 1)
    freq = frequencies(rot) if rot else None
    pos = torch.cat([torch.arange(p, p + n) for p, n in zip(pasts, lens)] + [torch.zeros(0, dtype=torch.int64)])
    kr, tk, qr, tq = k.double(), torch.zeros_like(k).double(), q.double(), torch.zeros_like(q).double()
    if rot:
        (kr, tk), (qr, tq) = attn_ref.rotate(k, pos, freq, halves), attn_ref.rotate(q, pos, freq, halves)
    want_k, want_v, tol = kc.double(), vc.double(), torch.zeros_like(kc).double()
    at = 0
    for s in range(b):
        for i in range(lens[s]):
            p = pasts[s] + i
            page_id, place = int(table[s, p // page]), p % page
            want_k[page_id, :, place], tol[page_id, :, place] = kr[at], tk[at]
            want_v[page_id, :, place] = v[at].double()
            at += 1
    dq, dk, dv = (x.to(DEV) if packed else x.to(DEV).unflatten(0, (b, lens[0])) for x in (q, k, v))
    kd, vd = kc.to(DEV), vc.to(DEV)
    k_out = torch.empty_like(dk)
    out = m3attn.m3_cache_append(dk, dv, kd, vd, table.to(DEV), torch.tensor(totals, dtype=torch.int32).to(DEV),
                                 q=dq if with_q else None, inv_freq=freq.to(DEV) if rot else None, halves=halves,
                                 cu_seqlens=torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV) if packed else None,
                                 k_out=k_out)
    torch.cuda.synchronize()
    assert_close(kd, want_k, tol, "k_cache")
    assert torch.equal(vd.cpu().double(), want_v)
    assert_close(k_out.reshape(k.shape), kr, tk, "k_out")
    if with_q:
        assert out.shape == dq.shape
        assert_close(out.reshape(q.shape), qr, tq, "q_out")
    else:
        assert out is None


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("d,rot", [(8, 8), (16, 0), (32, 32), (40, 40), (64, 16), (72, 72), (80, 32), (104, 24), (128, 128),
                                   (128, 64), (128, 8)])
def test_append_widths(io, halves, d, rot):
    check_append(io, [3, 0, 11, 1], [5, 9, 0, 30], 4, 2, d, 8, rot, halves, True, d + rot)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 256])
def test_append_pages(io, page):
    check_append(io, [1] * 5, [0, 1, 23, 24, 300], 6, 3, 64, page, 64, False, False, page)
    check_append(io, [50] * 2, [0, 31], 2, 2, 64, page, 64, True, False, page + 1)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (7, 7), (48, 8), (40, 1)])
def test_append_heads(io, hq, hk):
    check_append(io, [2, 5], [0, 4], hq, hk, 128, 16, 128, False, True, hq)
    check_append(io, [2, 5], [0, 4], hq, hk, 128, 16, 128, True, True, hq, with_q=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_append_far_positions(io):
    """Angles of a million radians: fp32 products of position and frequency would be off by 0.06."""
    d, page, pos = 64, 1 << 16, 1_048_573
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn(1, 1, 2, d, generator=g).to(IO[io]) for _ in range(2))
    kc = torch.zeros(1, 2, page, d, dtype=IO[io], device=DEV)
    table = torch.full((1, pos // page + 1), -1, dtype=torch.int32)
    table[0, -1] = 0
    lens = torch.tensor([pos + 1], dtype=torch.int32).to(DEV)
    freq = frequencies(d)
    out = m3attn.m3_cache_append(k.to(DEV), k.to(DEV), kc, torch.zeros_like(kc), table.to(DEV), lens, q=q.to(DEV),
                                 inv_freq=freq.to(DEV))
    torch.cuda.synchronize()
    want, tol = attn_ref.rotate(q[0], torch.tensor([pos]), freq, False)
    assert_close(out[0], want, tol, "q_out")
    want, tol = attn_ref.rotate(k[0], torch.tensor([pos]), freq, False)
    assert_close(kc[0, :, pos % page], want[0], tol[0], "k_cache")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("halves", [False, True])
def test_rotation_alone_and_back(io, halves):
    """In place, without a cache; turned frequencies undo it, and are its gradient."""
    g = torch.Generator().manual_seed(2)
    b, n, d = 2, 70, 64
    q, k = (torch.randn(b, n, h, d, generator=g).to(IO[io]) for h in (3, 1))
    freq = frequencies(48)
    qd, kd = q.to(DEV), k.to(DEV)
    out = m3attn.m3_cache_append(kd, None, q=qd, inv_freq=freq.to(DEV), halves=halves, q_out=qd, k_out=kd)
    torch.cuda.synchronize()
    assert out is qd
    pos = torch.arange(n).repeat(b)
    for got, x in ((qd, q), (kd, k)):
        want, tol = attn_ref.rotate(x.flatten(0, 1), pos, freq, halves)
        assert_close(got.flatten(0, 1), want, tol, "rotated")
    once = qd.cpu()
    m3attn.m3_cache_append(kd, None, q=qd, inv_freq=-freq.to(DEV), halves=halves, q_out=qd, k_out=kd)
    torch.cuda.synchronize()
    want, tol = attn_ref.rotate(once.flatten(0, 1), pos, -freq, halves)
    assert_close(qd.flatten(0, 1), want, tol, "back")
    half = torch.finfo(IO[io]).eps
    assert ((qd.cpu().double() - q.double()).abs() <= 2 * half * 2 * q.double().abs().amax(-1, keepdim=True)).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_append_strides(io):
    """Slices of one projection, caches of [pages, page_size, Hkv, D] in one buffer."""
    io = IO[io]
    g = torch.Generator().manual_seed(3)
    b, n, hq, hk, d, page = 2, 9, 4, 2, 64, 4
    wide = torch.randn(b, n, hq + 2 * hk + 1, d, generator=g).to(io).to(DEV)
    q, k, v = wide[:, :, :hq], wide[:, :, hq:hq + hk], wide[:, :, hq + hk:hq + 2 * hk]
    caches = torch.full((8, 2, page, hk, d), 7.0, dtype=io, device=DEV)
    kc, vc = caches[:, 0].transpose(1, 2), caches[:, 1].transpose(1, 2)
    table = torch.tensor([[6, 1, 4], [0, 7, 2]], dtype=torch.int32)
    freq = frequencies(d)
    before = wide.cpu()
    m3attn.m3_cache_append(k, v, kc, vc, table.to(DEV), None, q=q, inv_freq=freq.to(DEV), q_out=q, k_out=k)
    torch.cuda.synchronize()
    pos = torch.arange(n).repeat(b)
    want, tol = attn_ref.rotate(before[:, :, :hq].flatten(0, 1), pos, freq, False)
    assert_close(wide[:, :, :hq].flatten(0, 1), want, tol, "q in place")
    want, tol = attn_ref.rotate(before[:, :, hq:hq + hk].flatten(0, 1), pos, freq, False)
    assert_close(wide[:, :, hq:hq + hk].flatten(0, 1), want, tol, "k in place")
    assert torch.equal(wide[:, :, hq + hk:].cpu(), before[:, :, hq + hk:])
    got = caches.cpu()
    for s in range(b):
        for p in range(n):
            row = got[table[s, p // page], :, p % page]
            assert torch.equal(row[0], wide[s, p, hq:hq + hk].cpu()) and torch.equal(row[1], before[s, p, hq + hk:hq + 2 * hk])
    assert (got[3] == 7.0).all() and (got[5] == 7.0).all() and (got[4, :, 1:] == 7.0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("page", [4, 3])
def test_append_to_no_page(io, page):
    """Numbers that are no page, positions before 0 and past the table: not cached, everything else is."""
    d, hk = 32, 2
    kc = torch.full((5, hk, page, d), 7.0, dtype=IO[io], device=DEV)
    vc = kc.clone()
    table = torch.tensor([[-1, 2], [5, 1 << 30], [-(1 << 31), 4], [0, 1], [3, 3]], dtype=torch.int32)
    lens = torch.tensor([2 * page, 2 * page, 2 * page, 2 * page + 2, page - 1], dtype=torch.int32)
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(5, 2 * page, hk, d, generator=g).to(IO[io]) for _ in range(2))
    m3attn.m3_cache_append(k.to(DEV), v.to(DEV), kc, vc, table.to(DEV), lens.to(DEV))
    torch.cuda.synchronize()
    want_k, want_v = torch.full(kc.shape, 7.0, dtype=IO[io]), torch.full(kc.shape, 7.0, dtype=IO[io])
    for s in range(5):
        for i in range(2 * page):
            p = int(lens[s]) - 2 * page + i
            if 0 <= p < 2 * page and 0 <= int(table[s, p // page]) < 5:
                want_k[table[s, p // page], :, p % page], want_v[table[s, p // page], :, p % page] = k[s, i], v[s, i]
    assert torch.equal(kc.cpu(), want_k) and torch.equal(vc.cpu(), want_v)


def check_step(io, lens, hq, hk, d, page, seed, scale=None, bad=()):
    io = IO[io]
    kc, vc, table = make_cache(lens, hk, page, d, io, seed)
    g = torch.Generator().manual_seed(seed + 7)
    q = torch.randn(len(lens), hq, d, generator=g).to(io)
    keys, values = ([rows_of(c, table, s, n) for s, n in enumerate(lens)] for c in (kc, vc))
    ref = attn_ref.step(q, keys, values, scale)
    lse = torch.empty(len(lens), hq, device=DEV)
    o = m3attn.m3_attention_step(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV),
                                 torch.tensor(lens, dtype=torch.int32).to(DEV), scale, lse=lse)
    torch.cuda.synchronize()
    assert_close(o, ref["o"], ref["tol"]["o"], "o")
    some = torch.tensor(lens) > 0
    assert_close(lse[some.to(DEV)], ref["lse"][some], ref["tol"]["lse"][some], "lse")
    assert (lse[~some.to(DEV)] == float("-inf")).all()
    assert (o[~some.to(DEV)] == 0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("page", [1, 16, 24, 32, 64, 100])
def test_step_lengths(io, page):
    check_step(io, [0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 400, 0], 4, 2, 64, page, page)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [8, 16, 24, 40, 64, 72, 80, 96, 104, 120, 128])
@pytest.mark.parametrize("page", [32, 5])
def test_step_widths(io, d, page):
    check_step(io, [40, 0, 333, 1], 3, 1, d, page, d)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk", [(1, 1), (8, 8), (16, 1), (17, 1), (40, 1), (32, 8), (64, 2)])
def test_step_groups(io, hq, hk):
    check_step(io, [300, 70], hq, hk, 128, 16, hq + hk)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_long_and_short(io):
    """One sequence far longer than the others, cut into pieces that follow from all lengths."""
    check_step(io, [9000, 3, 0, 700, 256, 257, 1], 4, 1, 64, 64, 5)
    check_step(io, [20000], 2, 1, 128, 24, 6)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_many_sequences(io):
    """More sequences than lanes."""
    g = torch.Generator().manual_seed(10)
    check_step(io, torch.randint(0, 700, (150,), generator=g).tolist(), 2, 1, 32, 16, 11)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.01, 2.0])
def test_step_scales(io, scale):
    check_step(io, [1000, 50], 2, 2, 64, 16, 12, scale)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("page", [32, 7])
def test_step_shared_and_missing_pages(io, page):
    """Sequences that share pages; numbers that are no page leave their positions out; a length past the table is the
    table's; what lies behind a sequence's end, infinities and NaN included, is not looked at."""
    d, hk = 64, 2
    g = torch.Generator().manual_seed(13)
    kc, vc = (torch.randn(6, hk, page, d, generator=g).to(IO[io]) for _ in range(2))
    kc[5], vc[5] = float("nan"), float("inf")
    kc[4, :, 3:], vc[4, :, 3:] = float("inf"), float("nan")
    table = torch.tensor([[0, 1, 2], [0, 1, 4], [-1, 1, 6], [6, -5, 1 << 30], [3, 2, 1], [2, 5, 5]], dtype=torch.int32)
    lens = torch.tensor([3 * page, 2 * page + 3, 3 * page, 3 * page, 100 * page, page], dtype=torch.int32)
    q = torch.randn(6, 4, d, generator=g).to(IO[io])
    keys, values = [], []
    for s in range(6):
        there = [p for p in range(min(int(lens[s]), 3 * page)) if 0 <= int(table[s, p // page]) < 6]
        for out, c in ((keys, kc), (values, vc)):
            out.append(torch.stack([c[table[s, p // page], :, p % page] for p in there], 1) if there
                       else c.new_zeros(hk, 0, d))
    ref = attn_ref.step(q, keys, values)
    lse = torch.empty(6, 4, device=DEV)
    o = m3attn.m3_attention_step(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), lens.to(DEV), lse=lse)
    torch.cuda.synchronize()
    assert_close(o, ref["o"], ref["tol"]["o"], "o")
    assert (lse[3] == float("-inf")).all() and (o[3] == 0).all()
    keep = [0, 1, 2, 4, 5]
    assert_close(lse[keep], ref["lse"][keep], ref["tol"]["lse"][keep], "lse")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_no_cache(io):
    q = torch.ones(3, 2, 64, dtype=IO[io], device=DEV)
    empty = torch.empty(0, 1, 16, 64, dtype=IO[io], device=DEV)
    table = torch.zeros(3, 40, dtype=torch.int32, device=DEV)
    o = m3attn.m3_attention_step(q, empty, empty, table, torch.full((3,), 600, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert (o == 0).all()
    table = torch.zeros(3, 0, dtype=torch.int32, device=DEV)
    o = m3attn.m3_attention_step(q, empty, empty, table, torch.full((3,), 600, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert (o == 0).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_strides(io):
    """Queries as slices of a projection, in place; caches of [pages, page_size, Hkv, D] in one buffer."""
    io = IO[io]
    g = torch.Generator().manual_seed(14)
    b, hq, hk, d, page, lens = 3, 4, 2, 64, 32, [70, 300, 9]
    kc, vc, table = make_cache(lens, hk, page, d, io, 15)
    both = torch.stack([kc.transpose(1, 2), vc.transpose(1, 2)], 1).to(DEV)
    kd, vd = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    wide = torch.randn(b, hq + 3, d, generator=g).to(io).to(DEV)
    before = wide.cpu()
    keys, values = ([rows_of(c, table, s, n) for s, n in enumerate(lens)] for c in (kc, vc))
    ref = attn_ref.step(before[:, 1:1 + hq], keys, values)
    q = wide[:, 1:1 + hq]
    o = m3attn.m3_attention_step(q, kd, vd, table.to(DEV), torch.tensor(lens, dtype=torch.int32).to(DEV), o=q)
    torch.cuda.synchronize()
    assert o is q
    assert_close(q, ref["o"], ref["tol"]["o"], "o")
    assert torch.equal(wide[:, 0].cpu(), before[:, 0]) and torch.equal(wide[:, 1 + hq:].cpu(), before[:, 1 + hq:])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_step_of_infinities(io, bad):
    """What is attended to counts: an infinite value gives infinity, NaN gives NaN, in its column and sequence alone."""
    lens, d = [300, 80], 64
    kc, vc, table = make_cache(lens, 1, 16, d, IO[io], 16)
    vc[table[0, 2], 0, 5, 3] = bad
    q = torch.randn(2, 2, d, generator=torch.Generator().manual_seed(17)).to(IO[io])
    o = m3attn.m3_attention_step(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV),
                                 torch.tensor(lens, dtype=torch.int32).to(DEV)).cpu().float()
    assert (torch.isnan(o[0, :, 3]) if bad != bad else o[0, :, 3] == bad).all()
    o[0, :, 3] = 0
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_decoding_graph(io):
    """Append and step of one token, captured once and replayed while lengths grow, between eager work."""
    io = IO[io]
    b, hq, hk, d, page, steps = 3, 4, 2, 64, 16, 5
    starts = [40, 270, 0]
    kc, vc, table = make_cache([n + steps + 1 for n in starts], hk, page, d, io, 18)
    kd, vd, td, freq = kc.to(DEV), vc.to(DEV), table.to(DEV), frequencies(d).to(DEV)
    lens = torch.tensor(starts, dtype=torch.int32).to(DEV)
    k, v, q = (torch.zeros(b, 1, h, d, dtype=io, device=DEV) for h in (hk, hk, hq))

    def once():
        lens.add_(1)
        r = m3attn.m3_cache_append(k, v, kd, vd, td, lens, q=q, inv_freq=freq)
        return m3attn.m3_attention_step(r[:, 0], kd, vd, td, lens)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        once()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = once()
    lens.copy_(torch.tensor(starts, dtype=torch.int32))
    kd.copy_(kc), vd.copy_(vc)
    kr, vr, lr = kc.to(DEV), vc.to(DEV), lens.clone()
    g = torch.Generator().manual_seed(19)
    for _ in range(steps):
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=g).to(io))
        graph.replay()
        lr.add_(1)
        r = m3attn.m3_cache_append(k, v, kr, vr, td, lr, q=q, inv_freq=freq)
        want = m3attn.m3_attention_step(r[:, 0], kr, vr, td, lr)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(kd, kr) and torch.equal(vd, vr) and torch.equal(lens, lr)


def test_step_streams():
    """Two calls at once on two streams, with a workspace each, and again: equal bits."""
    lens = [5000, 900]
    kc, vc, table = make_cache(lens, 2, 16, 64, torch.bfloat16, 20)
    q = torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(21)).bfloat16().to(DEV)
    args = (kc.to(DEV), vc.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32).to(DEV))
    want = m3attn.m3_attention_step(q, *args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = [m3attn.m3_attention_step(q, *args, stream=s) for s in streams]
        for s in streams:
            s.synchronize()
        assert all(torch.equal(x, want) for x in got)


def test_large_cache():
    """Caches of 5 GB each: pages beyond 32 bits, appended to and read."""
    hk, hq, d, page, pages = 8, 16, 128, 64, 40000
    kd, vd = (torch.empty(pages, hk, page, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.tensor([[39999, 17], [20001, 39000]], dtype=torch.int32)
    n = 100
    g = torch.Generator().manual_seed(22)
    k, v = (torch.randn(2, n, hk, d, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(2, hq, d, generator=g).bfloat16()
    m3attn.m3_cache_append(k.to(DEV), v.to(DEV), kd, vd, table.to(DEV))
    o = m3attn.m3_attention_step(q.to(DEV), kd, vd, table.to(DEV), torch.full((2,), n, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    for s in range(2):
        for i in (0, 63, 64, 99):
            assert torch.equal(kd[table[s, i // page], :, i % page].cpu(), k[s, i])
    ref = attn_ref.step(q, [x.transpose(0, 1) for x in k], [x.transpose(0, 1) for x in v])
    assert_close(o, ref["o"], ref["tol"]["o"], "o")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("halves", [False, True])
def test_positions_below_32_bits(io, halves):
    """Lengths at int32's ends: positions lens - n + i beyond it are what they are, and are not cached."""
    g = torch.Generator().manual_seed(23)
    lens = torch.tensor([-(1 << 31), -(1 << 31) + 2, -5, 0, (1 << 31) - 1], dtype=torch.int32)
    b, n, d = len(lens), 4, 64
    q, k = (torch.randn(b, n, h, d, generator=g).to(IO[io]) for h in (3, 1))
    freq = frequencies(d) * 2.0 ** -9
    kc = torch.full((2, 1, 16, d), 7.0, dtype=IO[io], device=DEV)
    table = torch.zeros(b, 3, dtype=torch.int32, device=DEV)
    k_out = torch.empty_like(k.to(DEV))
    out = m3attn.m3_cache_append(k.to(DEV), k.to(DEV), kc, kc.clone(), table, lens.to(DEV), q=q.to(DEV), inv_freq=freq.to(DEV),
                                 halves=halves, k_out=k_out)
    torch.cuda.synchronize()
    pos = (lens.long().unsqueeze(1) - n + torch.arange(n)).flatten()
    assert int(pos.min()) < -(1 << 31)
    for got, x in ((out, q), (k_out, k)):
        want, tol = attn_ref.rotate(x.flatten(0, 1), pos, freq, halves)
        assert_close(got.flatten(0, 1), want, tol, "rotated")
    assert (kc == 7.0).all()
