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
