"""Checks of the attention kernels' assembly (no GPU needed): that of tests/test_mfma_hazards.py (no MFMA result is used
sooner after a taken branch than the compiler allows on straight-line code), waits before barriers, and register copies
that the compiler leaves under a partial execution mask."""
from __future__ import annotations

import re
import tempfile
from concurrent.futures import ThreadPoolExecutor

from test_mfma_hazards import WINDOW, _assembly, _distances, _split_kernels

SOURCES = ("attention.hip", "attention_backward.hip", "attention_step.hip")


def test_no_mfma_result_used_early_after_a_taken_branch():
    with tempfile.TemporaryDirectory() as d:
        with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
            paths = list(ex.map(lambda s: _assembly(s, d), SOURCES))
        kernels = [k for p in paths for k in _split_kernels(p)]
    straight, branched = {}, []
    for name, ins, labels in kernels:
        for op, dist, taken in _distances(ins, labels):
            if taken:
                branched.append((name, op, dist))
            else:
                straight[op] = min(straight.get(op, WINDOW), dist)
    assert straight, "no MFMA instruction found in the compiled kernels"
    bad = [(n, op, d, straight[op]) for n, op, d in branched if op in straight and d < straight[op]]
    assert not bad, "MFMA results used too early after a taken branch (kernel, opcode, distance, " \
                    "straight-line minimum): %s" % sorted(set(bad))[:10]


def _wait_before(ins, labels, i):
    """The loads that may still be on their way at barrier i: the vmcnt it waits for on straight line, with no load into
    LDS and no branch between; None: it does not."""
    targets, k = set(labels.values()), i
    while k > 0 and k not in targets:
        k -= 1
        o, oo = ins[k]
        if o == "s_waitcnt" and "vmcnt(" in " ".join(oo):
            return int(re.search(r"vmcnt\((\d+)\)", " ".join(oo)).group(1))
        if o.startswith(("s_cbranch", "s_branch", "s_barrier")) or (
                o.startswith("buffer_load") and any("lds" in x.split() for x in oo)):
            return None
    return None


def test_barriers_wait_for_loads_into_lds():
    """A wave's loads into LDS are counted by that wave alone, so each has to wait for its own before a barrier lets
    the others read.  Where tiles alternate every barrier waits for all; where two tiles take turns (few rows) one
    barrier of a round waits for all loads but the second tile's, and one for all."""
    with tempfile.TemporaryDirectory() as d:
        kernels = [k for s in SOURCES[:2] for k in _split_kernels(_assembly(s, d))]
    for name, ins, labels in kernels:
        waits = [_wait_before(ins, labels, i) for i, (op, _) in enumerate(ins) if op == "s_barrier"]
        assert waits or "_join" in name, name
        if "_few" not in name:
            assert all(w == 0 for w in waits), (name, waits)
            continue
        dim, size = (int(re.search(r"ELi(\d+)E|fLi(\d+)E", name).group(g) or 0) for g in (1, 2)), 2 if "bf16" in name else 4
        chunks = 128 * (64 if sum(dim) <= 64 else 128) * size // 16 // 256
        assert waits[0] is not None and waits[0] <= chunks and waits[1] == 0, (name, waits)


def _masked_copies(ins, labels):
    """Register copies and spills at the place where the lanes of a skipped region join again, before their bits of the
    execution mask are restored: lanes (or a whole wave) that skipped the region never get the copy."""
    found = []
    for label in sorted({oo[0] for o, oo in ins if o == "s_cbranch_execz"}):
        k, copies = labels.get(label, len(ins)), []
        while k < len(ins):
            o, oo = ins[k]
            if o.startswith("s_or_b64") and oo[:2] == ["exec", "exec"]:
                found += [(label, c) for c in copies]
                break
            if o.startswith(("s_cbranch", "s_branch", "s_endpgm", "s_setpc")) or "exec" in o or (oo and oo[0] == "exec"):
                break
            if o.startswith(("v_accvgpr", "scratch_")) or (o.startswith("v_mov_b") and oo[1][0] in "va"):
                copies.append(o + " " + ", ".join(oo))
            k += 1
    return found


def test_no_register_copy_before_the_mask_is_restored():
    with tempfile.TemporaryDirectory() as d:
        with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
            paths = list(ex.map(lambda s: _assembly(s, d), SOURCES))
        kernels = [k for p in paths for k in _split_kernels(p)]
    bad = [(name, c) for name, ins, labels in kernels for c in _masked_copies(ins, labels)]
    assert not bad, bad[:10]


def test_masked_copies_on_written_cases():
    region = [("s_and_saveexec_b64", ["s[0:1]", "vcc"]), ("s_cbranch_execz", [".L1"]), ("v_add_f32", ["v0", "v1", "v2"])]
    copy, restore = ("v_mov_b32_e32", ["v254", "v144"]), ("s_or_b64", ["exec", "exec", "s[0:1]"])
    at = {".L1": 3}
    assert _masked_copies(region + [copy, restore], at) == [(".L1", "v_mov_b32_e32 v254, v144")]
    assert _masked_copies(region + [("v_accvgpr_write_b32", ["a160", "v145"]), restore], at)
    assert not _masked_copies(region + [restore, copy], at)
    assert not _masked_copies(region + [("v_mov_b32_e32", ["v3", "0"]), restore], at)


def _fills(ins):
    """Loads into LDS in the order they are issued, as places in LDS ((unknown part, offset) of m0), and "|" for a
    barrier.  Scalar registers are followed in program order through what makes such places: a wave's part, shifted and
    added to, moves and spills."""
    val, spilled, out = {}, {}, []

    def read(t, at):
        if re.fullmatch(r"-?(0x[0-9a-f]+|\d+)", t):
            return (None, int(t, 0))
        return val.setdefault(t, (at, 0))

    for at, (op, oo) in enumerate(ins):
        if op == "s_barrier":
            out.append("|")
        elif op.startswith("buffer_load") and any("lds" in x.split() for x in oo):
            out.append(read("m0", at))
        elif op == "v_writelane_b32":
            spilled[oo[0], oo[2]] = read(oo[1], at)
        elif op == "v_readlane_b32":
            val[oo[0]] = spilled.get((oo[1], oo[2]), (at, 0))
        elif op.startswith(("s_", "v_readfirstlane")) and oo:
            made = None
            if op in ("s_mov_b32", "s_movk_i32"):
                made = read(oo[1], at)
            elif op in ("s_add_i32", "s_add_u32", "s_or_b32", "s_addk_i32"):
                a, b = [read(t, at) for t in (oo[1:3] if op != "s_addk_i32" else (oo[0], oo[1]))]
                if a[0] is None or b[0] is None:
                    made = (a[0] if b[0] is None else b[0], a[1] + b[1])
            pair = re.fullmatch(r"s\[(\d+):(\d+)\]", oo[0])
            for t in (["s%d" % i for i in range(int(pair.group(1)), int(pair.group(2)) + 1)] if pair else [oo[0]]):
                val[t] = made if made is not None and not pair else (at, 0)
    return out


def _tiles(fills, size):
    """Their tiles: 0 for the first one filled, 1 for the other; None: neither a tile nor whole rounds of one."""
    if not fills or any(f[0] != fills[0][0] for f in fills):
        return None
    low = min(f[1] for f in fills)
    tiles = [(f[1] - low) >= size for f in fills]
    if any(not 0 <= f[1] - low - t * (max(g[1] for g in fills) + 4096 - size - low) < size for f, t in zip(fills, tiles)):
        return None
    return [int(t != tiles[0]) for t in tiles]


def _run_order(fills, n):
    """The first n fills, then those of the loop behind them from its first barrier on: what stands before that is the
    loop's end, laid out at its top."""
    rest = fills[n:]
    first = rest.index("|") if "|" in rest else 0
    return fills[:n] + rest[first:] + rest[:first]


def test_tiles_are_filled_in_the_order_they_are_waited_for():
    """Few rows: the first barrier lets the second tile's loads be on their way, so those have to be the last ones issued,
    before the loop and in it, where the tile that is done with first is filled first again."""
    with tempfile.TemporaryDirectory() as d:
        kernels = [k for s in SOURCES[:2] for k in _split_kernels(_assembly(s, d)) if "_few" in k[0]]
    assert len(kernels) == 24
    for name, ins, _ in kernels:
        dim, size = (int(re.search(r"ELi(\d+)E|fLi(\d+)E", name).group(g) or 0) for g in (1, 2)), 2 if "bf16" in name else 4
        size *= 128 * (64 if sum(dim) <= 64 else 128)
        n = size // 16 // 256
        fills = _run_order(_fills(ins), 2 * n)
        tiles = _tiles([f for f in fills if f != "|"], size)
        assert tiles == [0] * n + [1] * n + [0] * n + [1] * n, (name, fills)
        assert fills[2 * n:2 * n + 2] == ["|", "|"] and fills[fills.index("|") + 1:].count("|") >= 2, (name, fills)
        loop = fills[2 * n:]
        assert "|" in loop[loop.index(next(f for f in loop if f != "|")) + n:][:1], (name, fills)   # between its tiles


def test_fill_order_on_written_cases():
    load, size = ("buffer_load_dwordx4", ["v1", "s[0:3]", "0 offen lds"]), 4096
    ins = [("s_lshl_b32", ["s5", "s4", "10"]), ("s_mov_b32", ["m0", "s5"]), load, ("s_add_i32", ["s6", "s5", "0x1000"]),
           ("v_writelane_b32", ["v9", "s6", "3"]), ("s_mov_b32", ["m0", "s6"]), load, ("s_barrier", []),
           ("s_mov_b32", ["s6", "s7"]), ("v_readlane_b32", ["s8", "v9", "3"]), ("s_mov_b32", ["m0", "s8"]), load,
           ("s_mov_b32", ["m0", "s5"]), load]
    fills = _fills(ins)
    assert [f[1] for f in fills if f != "|"] == [0, 4096, 4096, 0] and fills[2] == "|"
    assert _tiles([f for f in fills if f != "|"], size) == [0, 1, 1, 0]
    assert _run_order([1, 2, 5, "|", "|", 4, "|"], 2) == [1, 2, "|", "|", 4, "|", 5]
    assert _run_order([1, 2, "|", "|", 4, "|", 5], 2) == [1, 2, "|", "|", 4, "|", 5]
    assert _tiles(_fills([("s_mov_b32", ["m0", "s5"]), load, ("s_mov_b32", ["m0", "s6"]), load]), size) is None
