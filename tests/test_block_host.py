"""Host-side checks of include/m3block.h (no GPU needed): exports, structures, sizes, and every refusal with
its status and message.  Validation runs before any device access."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest
import torch

from state_space_sequence_m3_amd import m3block, m3scan

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "m3block.h")
P = ctypes.c_void_p
BASE, STRIDE = 0x10000, 1 << 32       # fake, aligned device addresses
NODEVICE = m3scan.M3_E_NODEVICE       # a valid call stops at the device check here


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(m3_[a-z_]+)\s*\(", text)))


def test_exports():
    lib = m3block.load()
    assert set(declared()) == set(m3block.EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", m3scan.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert set(declared()) <= set(re.findall(r"\bT\s+(m3_[a-z_]+)\b", out))
    assert all(hasattr(lib, n) for n in declared())


def test_structures_match_the_header(tmp_path):
    """Sizes and offsets as the C compiler sees them."""
    src = tmp_path / "sizes.cpp"
    fields = {"m3_scan_dims": m3block.M3ScanDims, "m3_norm_dims": m3block.M3NormDims,
              "m3_grad_tensor": m3block.M3GradTensor}
    lines = ['#include <cstdio>', '#include <cstddef>', '#include "m3block.h"', 'int main() {']
    want = []
    for name, cls in fields.items():
        lines.append('printf("%%zu\\n", sizeof(%s));' % name)
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append('printf("%%zu\\n", offsetof(%s, %s));' % (name, f))
            want.append(getattr(cls, f).offset)
    src.write_text("\n".join(lines + ["}"]))
    exe = str(tmp_path / "sizes")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    r = subprocess.run(["g++", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I",
                        os.path.join(rocm, "include"), str(src), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == want


def scan_dims(batch=2, seqlen=1000, width=130, io=m3block.M3_BF16, flags=0, **pitch):
    d = m3block.M3ScanDims(batch, seqlen, width, 0, 0, 0, 0, 0, io, flags)
    for k, v in pitch.items():
        setattr(d, k, v)
    return d


def norm_dims(rows=5, width=130, group=0, io=m3block.M3_BF16, flags=0, eps=1e-5, **pitch):
    d = m3block.M3NormDims(rows, width, 0, 0, 0, 0, 0, group, io, flags, eps)
    for k, v in pitch.items():
        setattr(d, k, v)
    return d


class Call:
    """One entry point with valid made-up pointers by name; arguments are replaced by keyword."""

    def __init__(self, fn, names, dims, ws_bytes=None):
        self.fn, self.names, self.dims, self.ws_bytes = fn, names, dims, ws_bytes

    def __call__(self, dims=None, ws_bytes=None, **kw):
        ptr = {n: BASE + i * STRIDE for i, n in enumerate(self.names)}
        ptr.update(kw)
        args = [P(ptr[n]) if ptr[n] else None for n in self.names]
        if self.ws_bytes is not None:
            args.append(self.ws_bytes if ws_bytes is None else ws_bytes)
        d = self.dims if dims is None else dims
        return getattr(m3block.load(), self.fn)(ctypes.byref(d) if d else None, *args, None)

    def addr(self, name):
        return BASE + self.names.index(name) * STRIDE


FWD = Call("m3_gated_scan", ["cu", "gate", "x", "bias", "h_in", "y", "h_out", "states", "ws"], scan_dims(), 1 << 30)
BWD = Call("m3_gated_scan_backward", ["cu", "gate", "x", "bias", "h_in", "states", "dy", "dh_out", "dgate", "dx",
                                      "dbias", "dh_in", "ws"], scan_dims(), 1 << 30)
STEP = Call("m3_gated_scan_step", ["gate", "x", "bias", "h", "y", "h_out"], scan_dims(seqlen=1))
NORM = Call("m3_rmsnorm", ["x", "residual", "weight", "r_out", "y", "q", "scale"], norm_dims())
NBWD = Call("m3_rmsnorm_backward", ["r", "weight", "dy", "dr_out", "dx", "dweight", "ws"], norm_dims(), 1 << 30)
ALL = [FWD, BWD, STEP, NORM, NBWD]

pytest_nodev = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU driver is present: made-up pointers "
                                  "must not get past the device check")


@pytest_nodev
@pytest.mark.parametrize("call", ALL, ids=lambda c: c.fn)
def test_valid_calls_stop_at_the_device(call):
    assert call() == NODEVICE


@pytest.mark.parametrize("call", ALL, ids=lambda c: c.fn)
def test_common_refusals(call):
    make = scan_dims if "scan" in call.fn else norm_dims
    one = {"seqlen": 1} if call is STEP else {}
    assert call(dims=make(io=5, **one)) == m3scan.M3_E_DTYPE
    assert call(dims=make(flags=1, **one)) == m3scan.M3_E_DIMS
    assert call(dims=make(width=-1, **one)) == m3scan.M3_E_DIMS
    fn = getattr(m3block.load(), call.fn)
    args = [None] * (len(fn.argtypes) - 1)
    if call.ws_bytes is not None:
        args[-2] = 0
    assert fn(None, *args) == m3scan.M3_E_NULL and "dims" in m3scan.last_error()


REQUIRED = [(FWD, n) for n in ("gate", "x", "y", "h_out")] + [(BWD, n) for n in ("gate", "x", "states", "dy", "dgate", "dx")] \
    + [(STEP, n) for n in ("gate", "x", "h", "y", "h_out")] + [(NORM, "x")] + [(NBWD, n) for n in ("r", "dy", "dx")]
OPTIONAL = [(FWD, n) for n in ("cu", "bias", "h_in", "states")] + [(BWD, n) for n in ("cu", "bias", "h_in", "dh_out",
                                                                                  "dbias", "dh_in")] \
    + [(STEP, "bias")] + [(NORM, n) for n in ("residual", "weight", "r_out", "y")] \
    + [(NBWD, n) for n in ("weight", "dr_out")]


@pytest.mark.parametrize("call,name", REQUIRED, ids=lambda v: getattr(v, "fn", v))
def test_required_pointers(call, name):
    assert call(**{name: 0}) == m3scan.M3_E_NULL
    assert name in m3scan.last_error()


@pytest_nodev
@pytest.mark.parametrize("call,name", OPTIONAL, ids=lambda v: getattr(v, "fn", v))
def test_optional_pointers(call, name):
    assert call(**{name: 0}) == NODEVICE


@pytest.mark.parametrize("call", ALL, ids=lambda c: c.fn)
def test_alignment(call):
    for name in call.names:
        if name == "q":
            continue
        off = 8 if name == "ws" else 1
        assert call(**{name: call.addr(name) + off}) == m3scan.M3_E_ALIGN, name


SAME_OK = {(FWD.fn, "h_out", "h_in"), (STEP.fn, "h_out", "h"), (STEP.fn, "y", "gate"), (STEP.fn, "y", "x"),
           (NORM.fn, "r_out", "x"), (NORM.fn, "r_out", "residual"), (NORM.fn, "y", "x"), (NORM.fn, "y", "residual"),
           (NBWD.fn, "dx", "dy"), (NBWD.fn, "dx", "dr_out")}
OUTS = {FWD.fn: ["y", "h_out", "states", "ws"], BWD.fn: ["dgate", "dx", "dbias", "dh_in", "ws"], STEP.fn: ["y", "h_out"],
        NORM.fn: ["r_out", "y", "q", "scale"], NBWD.fn: ["dx", "dweight", "ws"]}


@pytest_nodev
@pytest.mark.parametrize("call", ALL, ids=lambda c: c.fn)
def test_overlaps(call):
    """Every output against everything else: refused on top of it, and next to its start; allowed as the
    same buffer where the header says so."""
    for out in OUTS[call.fn]:
        for other in call.names:
            if other == out:
                continue
            on_top = call(**{out: call.addr(other)})
            ok = (call.fn, out, other) in SAME_OK
            assert on_top == (NODEVICE if ok else m3scan.M3_E_ALIAS), (out, other)
            if ok:
                near = 16
                assert call(**{out: call.addr(other) + near}) == m3scan.M3_E_ALIAS, (out, other)


@pytest_nodev
def test_slices_of_one_buffer():
    """Rows in each other's gaps are no overlap; one element more is."""
    d = scan_dims(width=64, y_pitch=200, gate_pitch=200, x_pitch=200)
    a = FWD.addr("gate")
    assert FWD(dims=d, x=a + 64 * 2, y=a + 128 * 2) == NODEVICE
    assert FWD(dims=d, x=a + 64 * 2, y=a + 127 * 2) == m3scan.M3_E_ALIAS     # into x
    assert FWD(dims=d, x=a + 64 * 2, y=a + 137 * 2) == m3scan.M3_E_ALIAS     # into gate's next row
    assert FWD(dims=d, x=a + 64 * 2, y=a + 136 * 2) == NODEVICE
    d.y_pitch = 201
    assert FWD(dims=d, x=a + 64 * 2, y=a + 128 * 2) == m3scan.M3_E_ALIAS     # other pitches cross
    d = norm_dims(width=64, r_pitch=128, y_pitch=128)
    a = NORM.addr("y")
    assert NORM(dims=d, r_out=a + 64 * 2) == NODEVICE
    assert NORM(dims=d, r_out=a + 62 * 2) == m3scan.M3_E_ALIAS


def test_pitches_and_sizes():
    for call, fields in ((FWD, ["gate_pitch", "x_pitch", "y_pitch"]), (BWD, ["dgate_pitch", "dx_pitch", "y_pitch"])):
        for f in fields:
            assert call(dims=scan_dims(**{f: 129})) == m3scan.M3_E_DIMS and f in m3scan.last_error()
            assert call(dims=scan_dims(**{f: 1 << 31})) == m3scan.M3_E_DIMS
    for f in ("x_pitch", "res_pitch", "r_pitch", "y_pitch"):
        assert NORM(dims=norm_dims(**{f: 100})) == m3scan.M3_E_DIMS
    assert NBWD(dims=norm_dims(dx_pitch=-1)) == m3scan.M3_E_DIMS
    big = (1 << 31) - 1
    assert FWD(dims=scan_dims(batch=big, seqlen=big), cu=0) == m3scan.M3_E_DIMS
    assert FWD(dims=scan_dims(batch=1 << 31)) == m3scan.M3_E_DIMS
    assert FWD(dims=scan_dims(batch=1, seqlen=1 << 30, x_pitch=big)) == m3scan.M3_E_DIMS
    assert FWD(dims=scan_dims(y_pitch=1 << 23)) == m3scan.M3_E_DIMS and "2^24" in m3scan.last_error()
    assert m3block.load().m3_gated_scan_workspace_bytes(ctypes.byref(scan_dims(batch=big, seqlen=big)), 0) == 0
    # a launch's threads: 2^23 blocks of 64 tokens and 128 channels are one too many
    many = {n: scan_dims(batch=1 << 22, seqlen=n, width=1) for n in (64, 65)}      # one and two blocks to a sequence
    rows = {n: m3block.load().m3_gated_scan_chunks(ctypes.byref(d), 0) for n, d in many.items()}
    assert rows == {64: 1 << 22, 65: 0}
    for call in (FWD, BWD):
        assert call(dims=many[65], cu=0) == m3scan.M3_E_DIMS and "2^23" in m3scan.last_error()
    assert STEP(dims=scan_dims(batch=1 << 16, width=1 << 15, seqlen=1)) == m3scan.M3_E_DIMS and "2^31" in m3scan.last_error()
    assert STEP(dims=scan_dims(seqlen=2)) == m3scan.M3_E_DIMS
    assert NORM(dims=norm_dims(width=16385)) == m3scan.M3_E_UNSUPPORTED
    assert NORM(dims=norm_dims(group=48)) == m3scan.M3_E_UNSUPPORTED
    assert NORM(dims=norm_dims(eps=-1.0)) == m3scan.M3_E_DIMS
    assert NORM(dims=norm_dims(eps=float("nan"))) == m3scan.M3_E_DIMS


def test_norm_outputs():
    assert NORM(y=0, q=0, scale=0) == m3scan.M3_E_NULL
    assert NORM(q=0) == m3scan.M3_E_NULL and "go together" in m3scan.last_error()
    assert NORM(scale=0) == m3scan.M3_E_NULL


def test_workspaces():
    lib = m3block.load()
    r = lambda n: (n + 255) // 256 * 256
    # `states` has a row per 64 tokens of a sequence (of the batch, where it is packed or its sequences are short and
    # many).  Chained tiles (forward 128 tokens, backward 64) need a 64-bit word per tile and channel (130 channels: 2
    # columns of 128) after 256 bytes, and marks where tiles hold several sequences; sequences of up to 2 tiles, and of
    # up to 8 where they fill the GPU with a workgroup each, are worked off without (fp32 forward: of one tile, if
    # few).  Backward also needs a row of partial sums per workgroup.
    words = lambda n: 256 + r(n * 256 * 8)
    row = 130 * 4
    marks = lambda t: r(-(-t // 64) * 16) + r(t * 4)       # where tiles hold several sequences: two bits and 4 bytes a token
    for kw, packed, rows, fwd16, fwd32, bwd in (
            (dict(), 0, 32, words(16), words(16), words(32) + 32 * row),
            (dict(), 1, 16, words(8) + marks(1000), words(8) + marks(1000), words(16) + marks(1000) + 16 * row),
            (dict(seqlen=300), 0, 10, words(6), words(6), words(10) + 10 * row),
            (dict(seqlen=300), 1, 5, words(3) + marks(300), words(3) + marks(300), words(5) + marks(300) + 5 * row),
            (dict(seqlen=256), 0, 8, 0, words(4), words(8) + 8 * row),
            (dict(seqlen=128), 0, 4, 0, 0, 2 * row),
            (dict(seqlen=128), 1, 2, 0, 0, words(2) + marks(128) + 2 * row),
            (dict(seqlen=64), 1, 1, 0, 0, 0),
            (dict(batch=256, seqlen=500), 0, 2048, 0, words(1024), 256 * row),               # 512 workgroups: a full round
            (dict(batch=256, seqlen=1000), 0, 4096, 0, words(2048), words(4096) + 4096 * row),
            (dict(batch=200, seqlen=1000), 0, 200 * 16, words(200 * 8), words(200 * 8), words(3200) + 3200 * row),
            (dict(batch=200, seqlen=3), 0, 200, 0, 0, 200 * row),
            (dict(batch=300, seqlen=3), 0, 15, words(8) + marks(900), words(8) + marks(900), words(15) + marks(900) + 15 * row),
            (dict(seqlen=0), 0, 1, 0, 0, 0), (dict(batch=0), 0, 1, 0, 0, 0)):
        for io in (m3block.M3_BF16, m3block.M3_F32):
            ref = ctypes.byref(scan_dims(io=io, **kw))
            assert lib.m3_gated_scan_chunks(ref, packed) == rows
            assert lib.m3_gated_scan_workspace_bytes(ref, packed) == (fwd16 if io == m3block.M3_BF16 else fwd32), kw
            assert lib.m3_gated_scan_backward_workspace_bytes(ref, packed) == bwd, kw
    for call in (FWD, BWD):
        need = getattr(lib, call.fn + "_workspace_bytes")(ctypes.byref(call.dims), 0)
        assert call(cu=0, ws_bytes=need - 1) == m3scan.M3_E_WORKSPACE
        assert call(cu=0, ws=0) == m3scan.M3_E_WORKSPACE
    need = lib.m3_rmsnorm_backward_workspace_bytes(ctypes.byref(norm_dims()))
    assert need > 0 and NBWD(ws_bytes=need - 1) == m3scan.M3_E_WORKSPACE
    assert lib.m3_rmsnorm_backward_workspace_bytes(ctypes.byref(norm_dims(rows=0))) == 0
    bad = scan_dims(width=-1)
    assert lib.m3_gated_scan_chunks(ctypes.byref(bad), 0) == 0 and lib.m3_gated_scan_chunks(None, 0) == 0
    if not os.path.exists("/dev/kfd"):
        assert NBWD(dweight=0, ws=0) == NODEVICE                   # nothing to sum: no workspace


def grad_call(name, entries, max_norm=1.0, stats=BASE + 90 * STRIDE, ws=BASE + 91 * STRIDE, ws_bytes=1 << 30, count=None):
    table = (m3block.M3GradTensor * max(1, len(entries)))()
    for t, (src, dst, n, io) in zip(table, entries):
        t.src, t.dst, t.numel, t.io = src, dst, n, io
    return getattr(m3block.load(), name)(ctypes.cast(table, P), len(entries) if count is None else count, max_norm,
                                         P(stats) if stats else None, P(ws) if ws else None, ws_bytes, None)


F, H = m3block.M3_F32, m3block.M3_BF16
A0, A1, A2 = BASE, BASE + STRIDE, BASE + 2 * STRIDE


@pytest.mark.parametrize("name", ["m3_grad_norm", "m3_grad_clip"])
def test_gradient_refusals(name):
    ok = [(A0, A0, 100000, F), (A1, A1, 50, H)]
    clip = name == "m3_grad_clip"
    assert grad_call(name, [(A0, A0, 100, 7)]) == m3scan.M3_E_DTYPE
    assert grad_call(name, [(A0, A0, -1, F)]) == m3scan.M3_E_DIMS
    assert grad_call(name, [(A0, A0, 1 << 40, F)]) == m3scan.M3_E_DIMS
    assert grad_call(name, ok, count=-1) == m3scan.M3_E_DIMS
    assert grad_call(name, [(None, A0, 1, F)]) == m3scan.M3_E_NULL
    assert grad_call(name, [(A0 + 2, A0 + 2, 10, F)]) == m3scan.M3_E_ALIGN
    assert grad_call(name, [(A0 + 1, A0 + 1, 10, H)]) == m3scan.M3_E_ALIGN
    assert grad_call(name, ok, max_norm=-1.0) == m3scan.M3_E_DIMS
    assert grad_call(name, ok, max_norm=float("nan")) == m3scan.M3_E_DIMS
    assert grad_call(name, ok, stats=0) == m3scan.M3_E_NULL
    assert grad_call(name, ok, stats=BASE + 90 * STRIDE + 2) == m3scan.M3_E_ALIGN
    assert grad_call(name, ok, ws=0) == m3scan.M3_E_WORKSPACE
    assert grad_call(name, ok, ws_bytes=63) == m3scan.M3_E_WORKSPACE        # 7 + 1 partial sums and their sum: 72
    assert grad_call(name, ok, ws=BASE + 91 * STRIDE + 8) == m3scan.M3_E_ALIGN
    assert grad_call(name, ok, stats=A0 + 8) == m3scan.M3_E_ALIAS
    assert grad_call(name, ok, ws=A1 + 32) == m3scan.M3_E_ALIAS
    assert grad_call(name, ok, stats=BASE + 91 * STRIDE + 8) == m3scan.M3_E_ALIAS
    if clip:
        assert grad_call(name, [(A0, None, 1, F)]) == m3scan.M3_E_NULL
        assert grad_call(name, [(A0, A0 + 8, 100, F)]) == m3scan.M3_E_ALIAS          # its own input in part
        assert grad_call(name, [(A0, A1, 100, F), (A0, A1, 100, F)]) == m3scan.M3_E_ALIAS
        assert grad_call(name, [(A0, A0, 100, F), (A0, A0, 100, F)]) == m3scan.M3_E_ALIAS
        assert grad_call(name, [(A0, A1, 100, F), (A1 + 396, A2, 5, F)]) == m3scan.M3_E_ALIAS
        assert grad_call(name, [(A1 + 396, A2, 5, F), (A0, A1, 100, F)]) == m3scan.M3_E_ALIAS
    if not os.path.exists("/dev/kfd"):
        assert grad_call(name, ok) == NODEVICE
        assert grad_call(name, [], ws=0) == NODEVICE
        assert grad_call(name, [(None, None, 0, F)], ws=0) == NODEVICE
        assert grad_call(name, [(A0, A1, 100, F), (A0, A2, 100, F)]) == NODEVICE     # one input, two outputs
        assert grad_call(name, [(A0, A0, 100, F), (A0 + 400, A0 + 400, 100, H)]) == NODEVICE


def test_gradient_workspace():
    lib = m3block.load()
    table = (m3block.M3GradTensor * 200)()
    for i, t in enumerate(table):
        t.src, t.dst, t.numel, t.io = A0 + i * 4096, A0 + i * 4096, 10, F
    size = lambda n: lib.m3_grad_workspace_bytes(ctypes.cast(table, P), n)
    assert size(0) == 0 and size(1) == 0 and size(96) == 0          # few elements: one workgroup, no partial sums
    assert size(200) == 201 * 8                                     # more tables than one
    table[0].numel = 65537
    assert size(1) == 6 * 8 and size(2) == 7 * 8
    table[0].numel = 16384 * 5000
    assert size(1) == 2049 * 8
    table[0].numel = 0
    assert size(1) == 0 and size(3) == 0
    assert lib.m3_grad_workspace_bytes(None, 3) == 0


def test_binding_checks():
    """What the binding refuses before it calls the library."""
    x = torch.zeros(2, 6, 8)
    with pytest.raises(ValueError, match="must be \\[b, L, D\\]"):
        m3block.m3_gated_scan(x[0], x[0])
    with pytest.raises(ValueError, match="shape"):
        m3block.m3_gated_scan(x[:, :5], x)
    with pytest.raises(ValueError, match="dtype"):
        m3block.m3_gated_scan(x.double(), x)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        m3block.m3_gated_scan(x.half(), x.half())
    with pytest.raises(ValueError, match="evenly spaced"):
        m3block.m3_gated_scan(torch.zeros(2, 9, 8)[:, :6], x)
    with pytest.raises(ValueError, match="dense and apart"):
        m3block.m3_gated_scan(x, torch.zeros(2, 6, 16)[..., ::2])
    with pytest.raises(ValueError, match="dense and apart"):
        m3block.m3_gated_scan(torch.zeros(8).expand(2, 6, 8), x)
    with pytest.raises(ValueError, match="bias"):
        m3block.m3_gated_scan(x, x, torch.zeros(7))
    with pytest.raises(ValueError, match="must be on a GPU"):
        m3block.m3_gated_scan(x, x)
    with pytest.raises(ValueError, match="cu_seqlens"):
        m3block.m3_gated_scan(x[0], x[0], cu_seqlens=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="contiguous"):
        m3block.m3_grad_clip([torch.zeros(4, 4).t()], 1.0)
    with pytest.raises(ValueError, match="outputs"):
        m3block.m3_grad_clip([x], 1.0, out=[])
    with pytest.raises(ValueError, match="must be on a GPU"):
        m3block.m3_rmsnorm(x)
    with pytest.raises(ValueError, match="weight"):
        m3block.m3_rmsnorm(x, weight=torch.zeros(9))
