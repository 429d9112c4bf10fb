"""m3_gated_scan, its backward pass and its single-token form against the formulas in 64 bits, at the
lengths, widths, layouts and batches where the tiles (128 tokens x 128 channels, 8 waves of 16 tokens)
can go wrong.  Bounds: tests/block_ref.py."""
from __future__ import annotations

import pytest
import torch

from block_ref import assert_close, offsets, scan
from state_space_sequence_m3_amd import m3block

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def draw(t, d, b, io, seed, bias=True, carry=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    return dict(gate=n(t, d).mul_(2).to(io), x=n(t, d).to(io), dy=n(t, d).to(io),
                bias=(torch.rand(d, generator=g) * -6) if bias else None,
                h_in=n(b, d) if carry else None, dh_out=n(b, d) if carry else None)


def dev(v):
    return None if v is None else v.to(DEV)


def run(c, lens, packed, layout="dense", tail=0):
    """Forward and backward on the GPU; returns outputs as [T, D] on the CPU."""
    t, d = c["x"].shape
    b, io = len(lens), c["x"].dtype
    gate, x, dy = dev(c["gate"]), dev(c["x"]), dev(c["dy"])
    kw = {}
    if layout == "sliced":     # gate and x as slices of one projection, gradients as slices of its gradient
        proj = torch.stack([gate, x], 1)
        gate, x = proj[:, 0], proj[:, 1]
        dproj = torch.full_like(proj, float("nan"))
        kw["grads"] = {"gate": dproj[:, 0], "x": dproj[:, 1]}
    elif layout == "odd":      # rows that start anywhere
        wide = torch.zeros(t, 2 * d + 5, dtype=io, device=DEV)
        wide[:, 1:d + 1], wide[:, d + 2:2 * d + 2] = gate, x
        gate, x = wide[:, 1:d + 1], wide[:, d + 2:2 * d + 2]
    if packed:
        extra = lambda v: torch.cat([v, torch.full((tail, d), float("nan"), dtype=io, device=DEV)]) if tail else v
        gate, x, dy = extra(gate), extra(x), extra(dy)
        cu = torch.tensor(offsets(lens), dtype=torch.int32, device=DEV)
    else:
        cu = None
        L = lens[0] if lens else 0
        gate, x, dy = (v.unflatten(0, (b, L)) for v in (gate, x, dy))
        if "grads" in kw:
            kw["grads"] = {k: v.unflatten(0, (b, L)) for k, v in kw["grads"].items()}
    bias, h_in, dh_out = dev(c["bias"]), dev(c["h_in"]), dev(c["dh_out"])
    marked = torch.full(x.shape, 7.0, dtype=io, device=DEV)
    y, h_out, states = m3block.m3_gated_scan(gate, x, bias, h_in, cu, y=marked, save_states=True)
    if tail and "grads" not in kw:
        kw["grads"] = {"gate": torch.full_like(marked, 7.0), "x": torch.full_like(marked, 7.0)}
    g = m3block.m3_gated_scan_backward(gate, x, dy, states, bias, h_in, dh_out, cu, **kw)
    torch.cuda.synchronize()
    if tail:                   # rows past the last sequence stay as they were
        for v in (y, g["gate"], g["x"]):
            assert (v[t:] == 7.0).all()
    flat = lambda v: v.reshape(-1, d)[:t].cpu()
    out = {"y": flat(y), "h_out": h_out.cpu(), "dgate": flat(g["gate"]), "dx": flat(g["x"])}
    if bias is not None:
        out["dbias"] = g["bias"].cpu()
    if h_in is not None:
        out["dh_in"] = g["h_in"].cpu()
    return out


def check(c, lens, got):
    ref = scan(c["gate"], c["x"], c["bias"], c["h_in"], lens, c["dy"], c["dh_out"])
    for k, v in got.items():
        assert_close(v, ref[k], ref["tol"][k], k)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("b,L,d", [(1, 1, 1), (1, 1, 128), (2, 15, 3), (3, 16, 130), (1, 17, 64), (2, 127, 256),
                                   (1, 128, 129), (2, 129, 128), (3, 300, 66), (1, 1300, 34), (40, 7, 257)])
def test_dense(io, b, L, d):
    c = draw(b * L, d, b, IO[io], seed=b * 1000 + L + d)
    check(c, [L] * b, run(c, [L] * b, packed=False))


@pytest.mark.parametrize("packed", [False, True])
def test_a_long_narrow_sequence(packed):
    """15000 tokens of 3 channels: all of the chain's tiles, over a hundred, run at the same time, so a tile's way back
    to a state can be as long as it may be.  Same bits every time."""
    c = draw(15000, 3, 1, torch.float32, 8)
    got = run(c, [15000], packed)
    check(c, [15000], got)
    for _ in range(3):
        again = run(c, [15000], packed)
        assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_workgroup_per_sequence(io):
    """As many sequences as fill the GPU are worked off one by one by their workgroups, without chains: sampled
    sequences against the formulas, the bias's gradient against that of the packed call, whose tiles are chained (each
    term off by at most 9 units per token, and the sums by their additions: 48 and one per 64 tiles)."""
    b, L, d = 512, 330, 130
    c = draw(b * L, d, b, IO[io], 17)
    got = run(c, [L] * b, packed=False)
    for s in (0, 200, 511):
        one = {k: (v if v is None or k == "bias" else v[s:s + 1] if k in ("h_in", "dh_out") else v[s * L:(s + 1) * L])
               for k, v in c.items()}
        ref = scan(one["gate"], one["x"], one["bias"], one["h_in"], [L], one["dy"], one["dh_out"])
        for k in ("y", "dgate", "dx"):
            assert_close(got[k][s * L:(s + 1) * L], ref[k], ref["tol"][k], k)
        for k in ("h_out", "dh_in"):
            assert_close(got[k][s:s + 1], ref[k], ref["tol"][k], k)
    other = run(c, [L] * b, packed=True)
    bound = 2 * got["dgate"].double().abs().sum(0) * (9 * L + 48 + b * L / 4096) * 2.0 ** -24
    assert ((got["dbias"].double() - other["dbias"].double()).abs() <= bound).all()


PACKED = [[1], [0], [0, 0, 5, 0], [128, 128], [127, 1, 129], [1] * 40, [3, 0, 250, 1, 0, 16, 400], [0, 513, 0]]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lens", PACKED, ids=lambda v: "-".join(map(str, v[:7])))
def test_packed(io, lens):
    c = draw(sum(lens), 70, len(lens), IO[io], seed=sum(lens) + len(lens))
    check(c, lens, run(c, lens, packed=True))
    check(c, lens, run(c, lens, packed=True, tail=150))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("most,carry", [(0, True), (1, True), (2, False), (3, True)])
def test_many_short_sequences(io, most, carry):
    """1300 sequences of up to `most` tokens, empty ones among them: more than the waves of a tile look through at
    once, and starts and ends at any place of a wave's tokens."""
    g = torch.Generator().manual_seed(most)
    lens = torch.randint(0, most + 1, (1300,), generator=g).tolist()
    c = draw(sum(lens), 70, len(lens), IO[io], seed=40 + most, carry=carry)
    check(c, lens, run(c, lens, packed=True, tail=3))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["sliced", "odd"])
@pytest.mark.parametrize("d", [128, 131])
def test_layouts(io, layout, d):
    c = draw(2 * 200, d, 2, IO[io], seed=d)
    check(c, [200, 200], run(c, [200, 200], packed=False, layout=layout))


@pytest.mark.parametrize("bias,carry", [(False, False), (True, False), (False, True)])
def test_optional_inputs(bias, carry):
    c = draw(2 * 150, 96, 2, torch.float32, 5, bias=bias, carry=carry)
    check(c, [150, 150], run(c, [150, 150], packed=False))


def test_no_tokens():
    """Empty sequences, dense or packed, pass the state and its gradient through; no sequences at all give a
    zero bias gradient."""
    h = torch.randn(3, 40, device=DEV)
    e = torch.empty(3, 0, 40, device=DEV)
    y, h_out, st = m3block.m3_gated_scan(e, e, None, h, save_states=True)
    g = m3block.m3_gated_scan_backward(e, e, e, st, torch.zeros(40, device=DEV), h, 2 * h)
    torch.cuda.synchronize()
    assert torch.equal(h_out, h) and torch.equal(g["h_in"], 2 * h) and not g["bias"].any()
    e = torch.empty(0, 40, device=DEV)
    cu = torch.zeros(1, dtype=torch.int32, device=DEV)
    y, h_out, st = m3block.m3_gated_scan(e, e, None, None, cu, save_states=True)
    g = m3block.m3_gated_scan_backward(e, e, e, st, torch.ones(40, device=DEV), cu_seqlens=cu)
    torch.cuda.synchronize()
    assert h_out.shape == (0, 40) and not g["bias"].any()


def test_extreme_gates():
    """Logits of +-infinity and of every size take x or keep h exactly."""
    d = 64
    u = torch.tensor([float("inf"), 200.0, 30.0, -30.0, -200.0, float("-inf")]).repeat(50)[:256]
    c = dict(gate=u.unsqueeze(1).repeat(1, d), x=torch.randn(256, d), dy=torch.randn(256, d), bias=None,
             h_in=torch.randn(1, d), dh_out=None)
    got = run(c, [256], packed=False)
    z, keep = torch.sigmoid(u.double()), torch.sigmoid(-u.double())
    h = c["h_in"][0].double()
    for t in range(256):
        h = keep[t] * h + z[t] * c["x"][t].double()
        assert torch.allclose(got["y"][t].double(), h, rtol=300 * 2.0 ** -24, atol=1e-30)
    for k in ("y", "dgate", "dx", "h_out"):
        assert torch.isfinite(got[k]).all()
    assert not got["dgate"][u.abs() == float("inf")].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_sequence_stays_alone(bad):
    """What a sequence holds never reaches its neighbours in a packed batch."""
    lens = [60, 200, 90, 300]
    c = draw(sum(lens), 64, 4, torch.float32, 11)
    clean = run(c, lens, packed=True)
    off = offsets(lens)
    for s in range(4):
        e = {k: (None if v is None else v.clone()) for k, v in c.items()}
        e["x"][off[s] + 5], e["dy"][off[s] + 9], e["h_in"][s], e["dh_out"][s] = bad, bad, bad, bad
        got = run(e, lens, packed=True)
        for k in ("y", "dgate", "dx"):
            for o in range(4):
                a, w = got[k][off[o]:off[o + 1]], clean[k][off[o]:off[o + 1]]
                assert torch.equal(a, w) == (o != s), (k, s, o)
        for o in range(4):
            for k in ("h_out", "dh_in"):
                assert torch.equal(got[k][o], clean[k][o]) == (o != s)


def test_offsets_that_break_the_rules_stay_in_bounds():
    """Offsets past T, negative or falling: no access leaves the buffers (rows outside keep their
    marks); results are unspecified."""
    d, t = 64, 300
    wide = torch.full((t + 200, d), 7.0, device=DEV)
    gate, x, dy = torch.randn(t, d, device=DEV), torch.randn(t, d, device=DEV), torch.randn(t, d, device=DEV)
    for cu in ([0, 100, 5000], [-7, 50, 300], [0, 250, 100], [10, 20, 30]):
        cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        y, h, st = m3block.m3_gated_scan(gate, x, cu_seqlens=cu, y=wide[100:100 + t], save_states=True)
        m3block.m3_gated_scan_backward(gate, x, dy, st, cu_seqlens=cu)
        torch.cuda.synchronize()
        assert (wide[:100] == 7.0).all() and (wide[100 + t:] == 7.0).all()


@pytest.mark.parametrize("t", [10, 300])
def test_tokens_without_a_sequence(t):
    """A packed batch of no sequences, with an end that breaks the rules: nothing is written but dbias, a sum of
    nothing."""
    x = torch.randn(t, 70, device=DEV)
    cu = torch.tensor([5], dtype=torch.int32, device=DEV)
    bias, none = torch.zeros(70, device=DEV), torch.zeros(0, 70, device=DEV)
    y, h, st = m3block.m3_gated_scan(x, x, bias, none, cu, y=torch.full_like(x, 7.0), save_states=True)
    g = m3block.m3_gated_scan_backward(x, x, x, st, bias, none, none, cu,
                                       grads={k: torch.full_like(x, 7.0) for k in ("gate", "x")})
    torch.cuda.synchronize()
    assert h.shape == g["h_in"].shape == (0, 70)
    assert all((v == 7.0).all() for v in (y, g["gate"], g["x"])) and (g["bias"] == 0).all()


def test_rows_four_gigabytes_apart():
    """Row offsets past 32 bits: 2100 tokens in a buffer of 2^20 elements per row (4.4 GB)."""
    t, d, pitch = 2100, 64, 1 << 20
    c = draw(t, d, 1, torch.bfloat16, 3)
    buf = torch.empty(t, pitch, dtype=torch.bfloat16, device=DEV)
    buf[:, 10:10 + d], buf[:, 200:200 + d], buf[:, 400:400 + d] = dev(c["gate"]), dev(c["x"]), dev(c["dy"])
    gate, x, dy = (buf[:, o:o + d].unsqueeze(0) for o in (10, 200, 400))
    y, h_out, st = m3block.m3_gated_scan(gate, x, dev(c["bias"]), dev(c["h_in"]), y=buf[:, 600:600 + d].unsqueeze(0),
                                         save_states=True)
    g = m3block.m3_gated_scan_backward(gate, x, dy, st, dev(c["bias"]), dev(c["h_in"]), dev(c["dh_out"]),
                                       grads={"gate": buf[:, 800:800 + d].unsqueeze(0),
                                              "x": buf[:, 1000:1000 + d].unsqueeze(0)})
    torch.cuda.synchronize()
    check(c, [t], {"y": y[0].cpu(), "h_out": h_out.cpu(), "dgate": g["gate"][0].cpu(), "dx": g["x"][0].cpu(),
                   "dbias": g["bias"].cpu(), "dh_in": g["h_in"].cpu()})


def test_state_in_place_and_calls_chained():
    """h_out may be h_in; a sequence cut over two calls gives what one call gives, up to rounding."""
    c = draw(700, 96, 1, torch.float32, 21)
    gate, x, bias = dev(c["gate"])[None], dev(c["x"])[None], dev(c["bias"])
    h = dev(c["h_in"]).clone()
    parts = [m3block.m3_gated_scan(gate[:, s], x[:, s], bias, h, h_out=h)[0]
             for s in (slice(0, 333), slice(333, 334), slice(334, 700))]
    torch.cuda.synchronize()
    ref = scan(c["gate"], c["x"], c["bias"], c["h_in"], [700])
    assert_close(torch.cat(parts, 1)[0], ref["y"], ref["tol"]["y"], "y")
    assert_close(h, ref["h_out"], ref["tol"]["h_out"], "h_out")


def test_equal_inputs_give_equal_bits():
    c = draw(8 * 1500, 256, 8, torch.bfloat16, 31)
    first = run(c, [1500] * 8, packed=False)
    for _ in range(5):
        again = run(c, [1500] * 8, packed=False)
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_gradients_against_differences():
    """Central differences of the 64-bit formula confirm the reference's gradients, which the tests
    above hold the kernels to."""
    lens, d = [5, 0, 9], 3
    c = draw(14, d, 3, torch.float32, 41)
    ref = scan(c["gate"], c["x"], c["bias"], c["h_in"], lens, c["dy"], c["dh_out"])

    def loss(e):
        r = scan(e["gate"], e["x"], e["bias"], e["h_in"], lens)
        return float((r["y"] * c["dy"].double()).sum() + (r["h_out"] * c["dh_out"].double()).sum())

    c64 = {k: (None if v is None else v.double()) for k, v in c.items()}
    for name, key in (("gate", "dgate"), ("x", "dx"), ("bias", "dbias"), ("h_in", "dh_in")):
        flat = c64[name].reshape(-1)
        for i in range(0, flat.numel(), 5):
            up, down = dict(c64), dict(c64)
            for e, s in ((up, 1e-5), (down, -1e-5)):
                e[name] = flat.clone()
                e[name][i] += s
                e[name] = e[name].view(c64[name].shape)
            slope = (loss(up) - loss(down)) / 2e-5
            assert abs(slope - float(ref[key].reshape(-1)[i])) < 1e-7


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("b,d", [(1, 1), (3, 5), (1, 64), (7, 132), (128, 1030), (2, 4096)])
@pytest.mark.parametrize("layout", ["dense", "sliced", "odd"])
def test_step(io, b, d, layout):
    c = draw(b, d, b, IO[io], seed=b + d)
    gate, x, h, bias = dev(c["gate"]), dev(c["x"]), dev(c["h_in"]), dev(c["bias"])
    if layout == "sliced":
        p = torch.stack([gate, x], 1)
        gate, x = p[:, 0], p[:, 1]
    elif layout == "odd":
        p = torch.cat([gate[:, :1], gate, x], 1)
        gate, x = p[:, 1:d + 1], p[:, d + 1:]
    ref = scan(c["gate"], c["x"], c["bias"], c["h_in"], [1] * b)
    h_new = torch.empty_like(h)
    y = m3block.m3_gated_scan_step(gate, x, h, bias, h_out=h_new)
    keep = h.clone()
    y2 = m3block.m3_gated_scan_step(gate, x, keep, bias)          # in place
    y3 = m3block.m3_gated_scan_step(gate, x.clone(), h, bias, y=x, h_out=torch.empty_like(h))   # y over x
    torch.cuda.synchronize()
    assert torch.equal(h, dev(c["h_in"])) and torch.equal(keep, h_new)
    assert torch.equal(y, y2) and torch.equal(y, y3)
    for got in (y, h_new):
        assert_close(got, ref["y"], ref["tol"]["y"], "step")


def test_steps_continue_a_scan():
    c = draw(20, 64, 1, torch.float32, 51)
    gate, x, bias = dev(c["gate"]), dev(c["x"]), dev(c["bias"])
    _, h = m3block.m3_gated_scan(gate[None, :12], x[None, :12], bias, dev(c["h_in"]))
    ys = [m3block.m3_gated_scan_step(gate[t:t + 1], x[t:t + 1], h, bias) for t in range(12, 20)]
    torch.cuda.synchronize()
    ref = scan(c["gate"], c["x"], c["bias"], c["h_in"], [20])
    assert_close(torch.cat(ys), ref["y"][12:], ref["tol"]["y"][12:], "steps")


def test_on_a_side_stream():
    """A call on a given stream allocates there and is ordered by it alone."""
    c = draw(600, 128, 1, torch.float32, 61)
    s = torch.cuda.Stream()
    args = [dev(c[k]) for k in ("gate", "x")]
    torch.cuda.synchronize()
    y, h = m3block.m3_gated_scan(args[0][None], args[1][None], dev(c["bias"]), dev(c["h_in"]), stream=s)
    s.synchronize()
    ref = scan(c["gate"], c["x"], c["bias"], c["h_in"], [600])
    assert_close(y[0], ref["y"], ref["tol"]["y"], "y")


def test_two_calls_at_once():
    """Chained calls on two streams, each with what it allocates, give what they give alone."""
    calls = []
    for seed, lens in ((1, [5000, 0, 1, 3000]), (2, [9000])):
        c = draw(sum(lens), 200, len(lens), torch.bfloat16, seed)
        a = {k: dev(v) for k, v in c.items()}
        calls.append((a, torch.tensor(offsets(lens), dtype=torch.int32, device=DEV)))

    def one(a, cu):
        y, h, st = m3block.m3_gated_scan(a["gate"], a["x"], a["bias"], a["h_in"], cu, save_states=True)
        g = m3block.m3_gated_scan_backward(a["gate"], a["x"], a["dy"], st, a["bias"], a["h_in"], a["dh_out"], cu)
        return [y, h, st] + [g[k] for k in sorted(g)]

    alone = [one(*c) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(one(*c))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(alone[i % 2], g))


def test_captured_and_replayed():
    """Forward and backward in one HIP graph, replayed on new inputs with eager calls in between."""
    t, d, b = 900, 192, 2
    bufs = {k: torch.zeros(b, t // b, d, device=DEV) for k in ("gate", "x", "dy")}
    bias = torch.randn(d, device=DEV) - 3
    h0 = torch.randn(b, d, device=DEV)

    def step():
        y, h, st = m3block.m3_gated_scan(bufs["gate"], bufs["x"], bias, h0, save_states=True)
        g = m3block.m3_gated_scan_backward(bufs["gate"], bufs["x"], bufs["dy"], st, bias, h0)
        return [y, h, g["gate"], g["x"], g["bias"], g["h_in"]]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(4):
        c = draw(t, d, b, torch.float32, 70 + seed)
        for k in bufs:
            bufs[k].copy_(c[k].view(b, t // b, d))
        graph.replay()
        torch.cuda.synchronize()
        kept = [v.clone() for v in captured]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for a, e in zip(kept, eager))


def test_one_workspace_for_calls_in_a_row():
    """A workspace needs no clearing: large, small and large again on the same memory."""
    ws = torch.full((8 << 20,), 0xab, dtype=torch.uint8, device=DEV)
    for t, d, seed in ((2000, 256, 1), (400, 64, 2), (2000, 256, 3)):
        c = draw(t, d, 1, torch.float32, seed)
        gate, x, dy = dev(c["gate"])[None], dev(c["x"])[None], dev(c["dy"])[None]
        y, h, st = m3block.m3_gated_scan(gate, x, dev(c["bias"]), save_states=True, workspace=ws)
        g = m3block.m3_gated_scan_backward(gate, x, dy, st, dev(c["bias"]), workspace=ws)
        torch.cuda.synchronize()
        ref = scan(c["gate"], c["x"], c["bias"], None, [t], c["dy"])
        assert_close(y[0], ref["y"], ref["tol"]["y"], "y")
        assert_close(g["gate"][0], ref["dgate"], ref["tol"]["dgate"], "dgate")
        assert_close(g["bias"], ref["dbias"], ref["tol"]["dbias"], "dbias")


def gates(gate, bias):
    """z and keep as the single-token form computes them, and the 64-bit logits, whose fp32 sums have to be exact."""
    d = gate.shape[1]
    u = gate.double() + bias.double()
    assert torch.equal(u, (gate.float() + bias).double())
    gate, bias = gate.to(DEV), bias.to(DEV)
    ones, zeros = torch.ones(gate.shape, device=DEV), torch.zeros(gate.shape, device=DEV)
    z, keep = torch.empty_like(ones), torch.empty_like(ones)
    m3block.m3_gated_scan_step(gate, ones.to(gate.dtype), zeros, bias, h_out=z)        # 0 keep + 1 z
    m3block.m3_gated_scan_step(gate, zeros.to(gate.dtype), ones, bias, h_out=keep)     # 1 keep + 0 z
    torch.cuda.synchronize()
    return z.cpu().double(), keep.cpu().double(), u


def draw_gates(io, cancel):
    """Logits of up to 70 on a grid of 2^-7 that bf16 and fp32 both hold: gate a whole number from -256 to 256, bias
    with a fraction, where they cancel of the other sign."""
    g = torch.Generator().manual_seed(9)
    bias = torch.randint(-2 ** 14, 2 ** 14, (512,), generator=g) / 128.0
    gate = torch.randint(-70, 71, (2000, 512), generator=g).float()
    gate = (gate - bias.round() if cancel else gate).clamp(-256, 256)
    if not cancel:
        bias = bias / 64
    return gate.to(IO[io]), bias


@pytest.mark.parametrize("cancel", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_both_gates_keep_their_digits(io, cancel):
    """In units of 2^-24: e^-|u| is off by 2 for the exponential (one step of its last place) and 1 for the product that
    carries the rest, its sum with 1 by 1, the reciprocal by 2 (one step), the product by 1: both gates by at most 7."""
    z, keep, u = gates(*draw_gates(io, cancel))
    for got, ref in ((z, torch.sigmoid(u)), (keep, torch.sigmoid(-u))):
        assert ((got - ref).abs() <= 7.1 * 2.0 ** -24 * ref).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_the_larger_gate_is_rounded_once(io):
    """big = 1 / (1 + e) in units of 2^-24, its own half step being 1/2: the sum's rounding moves it by big^2, e's error of
    3 by 3 e big^2; a reciprocal that is not the nearest would add to that, always to one side, token after token.  1e-3 covers products of errors,
    which are 2^-22 of one."""
    g = torch.Generator().manual_seed(10)
    if io == "f32":
        gate, bias = (torch.rand(4000, 512, generator=g) - 0.5) * 40, torch.zeros(512)
    else:                    # many values of one type's few: gates of whole numbers, biases with fractions of 2^-16
        gate = torch.randint(-10, 11, (4000, 512), generator=g).to(torch.bfloat16)
        bias = torch.randint(-2 ** 20, 2 ** 20, (512,), generator=g) / 2.0 ** 16
    z, keep, u = gates(gate, bias)
    e = torch.exp(-u.abs())
    big = 1 / (1 + e)
    got = torch.where(u >= 0, z, keep)
    assert ((got - big).abs() <= (0.5 + big * big * (1 + 3 * e) + 1e-3) * 2.0 ** -24).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("b,L,d", [(700, 7, 70), (300, 3, 257), (520, 64, 66), (513, 1, 5)])
def test_many_short_dense_sequences(io, b, L, d):
    """Dense sequences of up to 64 tokens, too many for a workgroup each, share tiles.  The reference runs them side by
    side as channels of one sequence; the bias's gradient adds up over them (its additions: block_ref)."""
    assert b * -(-d // 128) > 512
    c = draw(b * L, d, b, IO[io], seed=b + L + d)
    got = run(c, [L] * b, packed=False)
    side = lambda v: v.view(b, L, d).transpose(0, 1).reshape(L, b * d)
    flat = lambda v: None if v is None else v.reshape(1, b * d)
    ref = scan(side(c["gate"]), side(c["x"]), c["bias"].repeat(b), flat(c["h_in"]), [L], side(c["dy"]), flat(c["dh_out"]))
    for k in ("y", "dgate", "dx"):
        assert_close(side(got[k]), ref[k], ref["tol"][k], k)
    for k in ("h_out", "dh_in"):
        assert_close(flat(got[k]), ref[k], ref["tol"][k], k)
    over = lambda v: v.view(b, d).sum(0)
    assert_close(got["dbias"], over(ref["dbias"]), over(ref["tol"]["dbias"]) + over(ref["dgate"].abs().sum(0)) *
                 (48 + b * L / 4096) * 2.0 ** -24, "dbias")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("b,L,d", [(5, 700, 66), (7, 1100, 130)])
def test_chains_side_by_side(io, b, L, d):
    """Tiles of four sequences are taken in turns, then those of the rest: of one, and of three."""
    c = draw(b * L, d, b, IO[io], seed=b + L + d)
    check(c, [L] * b, run(c, [L] * b, packed=False))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gates_at_the_ends(io):
    """Infinite and far logits give gates of 0 and 1 exactly, also with a bias that ends there; NaN stays NaN."""
    inf, nan = float("inf"), float("nan")
    gate = torch.tensor([[inf, -inf, 200.0, -200.0, nan, 0.0, inf, 1.0, -1.0, 3e38]]).to(IO[io]).repeat(3, 1).to(DEV)
    bias = torch.tensor([0.0, 0.0, 0.0, 0.0, 0.0, nan, -inf, inf, -inf, 3e38], device=DEV)
    want = torch.tensor([1.0, 0.0, 1.0, 0.0, nan, nan, nan, 1.0, 0.0, 1.0])
    ones, z = torch.ones(3, 10, device=DEV), torch.empty(3, 10, device=DEV)
    m3block.m3_gated_scan_step(gate, ones.to(IO[io]), 0 * ones, bias, h_out=z)
    _, last = m3block.m3_gated_scan(gate[None], ones.to(IO[io])[None], bias, torch.zeros(1, 10, device=DEV))
    torch.cuda.synchronize()
    for row in z.cpu():
        assert torch.equal(row.isnan(), want.isnan()) and torch.equal(row.nan_to_num(), want.nan_to_num())
    assert torch.equal(last[0].cpu().nan_to_num(), want.nan_to_num()) and torch.equal(last[0].cpu().isnan(), want.isnan())
