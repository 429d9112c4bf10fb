"""Host-side checks of include/m3attn.h (no GPU needed): exports, structures, sizes, every refusal with its status and
message, the index maps of the kernels compiled for the host (bad pages among them), and the binding's own
checks.  Validation runs before any device access."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest
import torch

from state_space_sequence_m3_amd import m3attn, m3scan

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "m3attn.h")
P = ctypes.c_void_p
BASE, STRIDE = 0x10000, 1 << 36       # fake, aligned device addresses
NODEVICE = m3scan.M3_E_NODEVICE       # a valid call stops at the device check here
DENSE = (0, 0, 0)

pytest_nodev = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU driver is present: made-up pointers "
                                  "must not get past the device check")


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(m3_[a-z_]+)\s*\(", text)))


def test_exports():
    lib = m3attn.load()
    assert set(declared()) == set(m3attn.EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", m3scan.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert set(declared()) <= set(re.findall(r"\bT\s+(m3_[a-z_]+)\b", out))
    assert all(hasattr(lib, n) for n in declared())


def test_structures_match_the_header(tmp_path):
    """Sizes and offsets as the C compiler sees them."""
    src = tmp_path / "sizes.cpp"
    lines = ['#include <cstdio>', '#include <cstddef>', '#include "m3attn.h"', 'int main() {']
    want = []
    for name, cls in {"m3_attn_dims": m3attn.M3AttnDims, "m3_cache_dims": m3attn.M3CacheDims}.items():
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


MAPS = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "m3_page_map.h"
using namespace m3;
static unsigned long long state = 88172645463325252ull;
static long rnd(long n) { state ^= state << 13; state ^= state >> 7; state ^= state << 17; return (long)(state % (unsigned long long)n); }
#define CHECK(c) do { if (!(c)) { std::printf("line %d\n", __LINE__); return 1; } } while (0)
int main() {
    // pages: powers of two and not, the ends of the table, numbers that are no page, negative positions
    const int32_t table[5] = {3, -1, 7, 0, 8};
    for (int32_t size : {1, 2, 7, 16, 24, 64}) {
        int shift = -1;
        for (int i = 0; i < 31; ++i) if (size == 1 << i) shift = i;
        for (int s : {-1, shift})
            for (int32_t pos = -3; pos < 7 * size; ++pos) {
                int32_t place = 99;
                const int32_t id = page_place(table, 5, 8, size, s, pos, &place);
                if (pos < 0 || pos >= 5 * size) { CHECK(id == -1); continue; }
                const int32_t want = table[pos / size];
                CHECK(id == (want >= 0 && want < 8 ? want : -1));
                CHECK(place == pos % size);
            }
        int32_t place;
        CHECK(page_place(table, 5, 8, size, shift, 0x7fffffff, &place) == -1);
        CHECK(page_place(table, 5, 8, size, shift, (int32_t)0x80000000, &place) == -1);
        CHECK(page_place(table, 0, 8, size, shift, 0, &place) == -1);
        CHECK(page_place(table, 5, 0, size, shift, 0, &place) == -1);
    }
    // blocks of a packed batch: every row of every sequence in exactly one block, numbers within T / R + b
    for (int round = 0; round < 300; ++round) {
        const long b = 1 + rnd(90), R = 128, most = 1 + rnd(600);
        std::vector<long> cu(b + 1, 0);
        for (long s = 0; s < b; ++s) cu[s + 1] = cu[s] + (rnd(3) ? rnd(most) : 0);
        const long T = cu[b] + rnd(200), blocks = T / R + b;
        std::vector<int> seen(T, 0);
        for (long n = 0; n < blocks; ++n) {
            long s = 0;
            for (long i = 0; i < b; ++i) if (first_block(cu[i], i, R) <= n) s = i;
            const long r0 = (n - first_block(cu[s], s, R)) * R;
            CHECK(r0 >= 0);
            for (long r = r0; r < r0 + R && r < cu[s + 1] - cu[s]; ++r) seen[cu[s] + r]++;
        }
        for (long t = 0; t < T; ++t) CHECK(seen[t] == (t < cu[b] ? 1 : 0));
    }
    // the order of workgroups: a permutation that keeps each on its XCD
    for (long n = 1; n <= 2000; ++n) {
        std::vector<int> seen(n, 0);
        for (long i = 0; i < n; ++i) {
            const long j = (long)paired_item(i, n);
            CHECK(j >= 0 && j < n && !seen[j]++ && j % kXcds == i % kXcds);
            CHECK(j == i || (i >= kUnits && i < 2 * kUnits));
        }
    }
    // pieces of a decoding batch: at most `items`, whole rounds, and numbers piece + sequence of their parts all
    // different, those of a sequence in a row, below items + b
    for (int round = 0; round < 2000; ++round) {
        const long b = 1 + rnd(200), items = 1 + rnd(2000), most = 1 + rnd(100000);
        std::vector<long> start(b + 1, 0);
        for (long s = 0; s < b; ++s) {
            const long len = rnd(3) ? rnd(most) : 0, n = rounded_keys(len);
            CHECK(n >= kRound && n % kRound == 0 && n >= len && (n == kRound || n - kRound < len));
            start[s + 1] = start[s] + n;
        }
        const long keys = piece_keys(start[b], items), pieces = (start[b] + keys - 1) / keys;
        CHECK(keys >= kRound && keys % kRound == 0 && pieces <= items);
        std::vector<int> seen(items + b, 0);
        for (long s = 0; s < b; ++s)
            for (long i = start[s] / keys; i <= (start[s + 1] - 1) / keys; ++i) {
                CHECK(i < pieces && i + s < items + b);
                CHECK(!seen[i + s]++);
            }
    }
    std::printf("ok\n");
    return 0;
}
"""


def test_index_maps(tmp_path):
    src, exe = tmp_path / "maps.cpp", str(tmp_path / "maps")
    src.write_text(MAPS)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I",
                        os.path.join(ROOT, "state_space_sequence_m3_amd", "csrc"), str(src), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr


def attn_dims(batch=2, seqlen=300, heads=8, kv_heads=2, head_dim=64, io=m3attn.M3_BF16, flags=0, scale=0.0, **strides):
    d = m3attn.M3AttnDims(batch, seqlen, heads, kv_heads, head_dim, *[DENSE] * 8, io, flags, scale)
    for k, v in strides.items():
        setattr(d, k, v)
    return d


def cache_dims(batch=3, seqlen=1, heads=8, kv_heads=2, head_dim=64, num_pages=50, page_size=16, table_width=40, rotary_dim=0,
               io=m3attn.M3_BF16, flags=0, scale=0.0, **strides):
    d = m3attn.M3CacheDims(batch, seqlen, heads, kv_heads, head_dim, num_pages, page_size, table_width, rotary_dim,
                           *[DENSE] * 8, io, flags, scale)
    for k, v in strides.items():
        setattr(d, k, v)
    return d


class Call:
    """One entry point with valid made-up pointers by name; arguments are replaced by keyword."""

    def __init__(self, fn, names, make, ws_bytes=None, **usual):
        self.fn, self.names, self.ws_bytes = fn, names, ws_bytes
        self.make = lambda **kw: make(**{**usual, **kw})

    def __call__(self, dims=None, ws_bytes=None, **kw):
        ptr = {n: BASE + i * STRIDE for i, n in enumerate(self.names)}
        ptr.update(kw)
        args = [P(ptr[n]) if ptr[n] else None for n in self.names]
        if self.ws_bytes is not None:
            args.append(self.ws_bytes if ws_bytes is None else ws_bytes)
        return getattr(m3attn.load(), self.fn)(ctypes.byref(self.make() if dims is None else dims), *args, None)

    def addr(self, name):
        return BASE + self.names.index(name) * STRIDE


FWD = Call("m3_attention", ["cu", "q", "k", "v", "o", "lse"], attn_dims)
BWD = Call("m3_attention_backward", ["cu", "q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv", "workspace"], attn_dims, 1 << 30)
APP = Call("m3_cache_append", ["cu", "lens", "inv_freq", "q", "k", "v", "q_out", "k_out", "k_cache", "v_cache", "page_table"],
           cache_dims, seqlen=20, rotary_dim=32)
STEP = Call("m3_attention_step", ["q", "k_cache", "v_cache", "page_table", "lens", "o", "lse", "workspace"], cache_dims, 1 << 30)
ALL = [FWD, BWD, APP, STEP]
BY = lambda v: getattr(v, "fn", v)


@pytest_nodev
@pytest.mark.parametrize("call", ALL, ids=BY)
def test_valid_calls_stop_at_the_device(call):
    assert call() == NODEVICE


@pytest.mark.parametrize("call", ALL, ids=BY)
def test_common_refusals(call):
    for field, value, status in [("io", 5, m3scan.M3_E_DTYPE), ("flags", 4, m3scan.M3_E_DIMS), ("batch", -1, m3scan.M3_E_DIMS),
                                 ("batch", 1 << 31, m3scan.M3_E_DIMS), ("seqlen", -1, m3scan.M3_E_DIMS),
                                 ("heads", 0, m3scan.M3_E_DIMS), ("kv_heads", 0, m3scan.M3_E_DIMS),
                                 ("kv_heads", 3, m3scan.M3_E_DIMS), ("kv_heads", -2, m3scan.M3_E_DIMS),
                                 ("heads", 1 << 21, m3scan.M3_E_DIMS), ("head_dim", 0, m3scan.M3_E_DIMS),
                                 ("head_dim", 60, m3scan.M3_E_DIMS), ("head_dim", 136, m3scan.M3_E_UNSUPPORTED)]:
        assert call(dims=call.make(**{field: value})) == status, field
    fn = getattr(m3attn.load(), call.fn)
    args = [None] * (len(fn.argtypes) - 1)
    if call.ws_bytes is not None:
        args[-2] = 0
    assert fn(None, *args) == m3scan.M3_E_NULL and "dims" in m3scan.last_error()


@pytest.mark.parametrize("call", [FWD, BWD, STEP], ids=BY)
def test_scales(call):
    for bad in (-1.0, float("nan"), float("inf")):
        assert call(dims=call.make(scale=bad)) == m3scan.M3_E_DIMS and "scale" in m3scan.last_error()


REQUIRED = [(FWD, n) for n in ("q", "k", "v", "o")] + [(BWD, n) for n in ("q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv")] \
    + [(APP, n) for n in ("inv_freq", "q", "k", "v", "q_out", "k_cache", "v_cache", "page_table")] \
    + [(STEP, n) for n in ("q", "k_cache", "v_cache", "page_table", "lens", "o")]
OPTIONAL = [(FWD, n) for n in ("cu", "lse")] + [(BWD, "cu")] + [(APP, n) for n in ("cu", "lens", "k_out")] + [(STEP, "lse")]


@pytest.mark.parametrize("call,name", REQUIRED, ids=BY)
def test_required_pointers(call, name):
    assert call(**{name: 0}) == m3scan.M3_E_NULL
    assert name in m3scan.last_error()


@pytest_nodev
@pytest.mark.parametrize("call,name", OPTIONAL, ids=BY)
def test_optional_pointers(call, name):
    assert call(**{name: 0}) == NODEVICE


@pytest_nodev
def test_append_without_queries_or_caches():
    assert APP(q=0, q_out=0) == NODEVICE
    assert APP(k_cache=0, v_cache=0, page_table=0) == NODEVICE
    assert APP(k_cache=0, v_cache=0, page_table=0, v=0) == NODEVICE
    assert APP(inv_freq=0, dims=APP.make(rotary_dim=0)) == NODEVICE


@pytest.mark.parametrize("call", ALL, ids=BY)
def test_alignment(call):
    for name in call.names:
        off = 2 if name in ("cu", "lens", "inv_freq", "page_table", "lse") else 8
        assert call(**{name: call.addr(name) + off}) == m3scan.M3_E_ALIGN, name
        if off == 8:
            assert name in m3scan.last_error()


STRIDED = [(FWD, n, 300) for n in ("q", "k", "v", "o")] + [(BWD, n, 300) for n in ("dout", "dq", "dk", "dv")] \
    + [(APP, n, 20) for n in ("q", "k", "v", "q_out", "k_out")]


@pytest.mark.parametrize("call,name,n", STRIDED, ids=BY)
def test_strides(call, name, n):
    wide = 64 * 8 * 4
    usual = [n * wide, wide, 64]
    assert call(dims=call.make(**{name: (usual[0], usual[1], 60)})) == m3scan.M3_E_ALIGN and name in m3scan.last_error()
    assert call(dims=call.make(**{name: (usual[0], usual[1] + 4, 64)})) == m3scan.M3_E_ALIGN
    assert call(cu=0, dims=call.make(**{name: (usual[0] + 4, usual[1], 64)})) == m3scan.M3_E_ALIGN
    assert call(cu=0, dims=call.make(**{name: (-8, usual[1], 64)})) == m3scan.M3_E_DIMS
    assert call(dims=call.make(**{name: (usual[0], -8, 64)})) == m3scan.M3_E_DIMS
    assert call(cu=0, dims=call.make(**{name: (1 << 48, usual[1], 64)})) == m3scan.M3_E_DIMS
    assert call(dims=call.make(**{name: (n << 23, 1 << 23, 64)})) == m3scan.M3_E_DIMS and "2^24" in m3scan.last_error()


@pytest_nodev
@pytest.mark.parametrize("call,name,n", STRIDED, ids=BY)
def test_strides_that_are_taken(call, name, n):
    wide = 64 * 8 * 4
    assert call(dims=call.make(**{name: (n * wide, wide, 64)})) == NODEVICE
    assert call(cu=0, dims=call.make(**{name: (n * 64 * 8, 64, n * 64)})) == NODEVICE         # heads before tokens
    out = name in ("o", "dq", "dk", "dv", "q_out", "k_out")
    assert call(dims=call.make(**{name: (n * wide, wide, 0)})) == (m3scan.M3_E_ALIAS if out else NODEVICE)
    assert call(dims=call.make(**{name: (0, wide, 64)})) == NODEVICE                         # packed: not used
    assert call(cu=0, dims=call.make(**{name: (0, wide, 64)})) == (m3scan.M3_E_ALIAS if out else NODEVICE)
    assert call(dims=call.make(**{name: (n * wide, 32, 64)})) == (m3scan.M3_E_ALIAS if out else NODEVICE)


OUTS = {FWD.fn: ["o", "lse"], BWD.fn: ["dq", "dk", "dv", "workspace"], APP.fn: ["q_out", "k_out", "k_cache", "v_cache"],
        STEP.fn: ["o", "lse", "workspace"]}
SAME_OK = {(APP.fn, "q_out", "q"), (APP.fn, "k_out", "k"), (STEP.fn, "o", "q")}


@pytest_nodev
@pytest.mark.parametrize("call", ALL, ids=BY)
def test_overlaps(call):
    """Every output against everything else: refused on top of it, and next to its start; allowed as the same buffer where
    the header says so."""
    for out in OUTS[call.fn]:
        for other in call.names:
            if other == out:
                continue
            ok = (call.fn, out, other) in SAME_OK
            assert call(**{out: call.addr(other)}) == (NODEVICE if ok else m3scan.M3_E_ALIAS), (out, other)
            if ok:
                assert call(**{out: call.addr(other) + 16}) == m3scan.M3_E_ALIAS, (out, other)
                other_strides = {"q_out" if call is APP and out == "q_out" else out: (64 * 8 * 20 * 2, 64 * 8 * 2, 64)}
                assert call(dims=call.make(**other_strides), **{out: call.addr(other)}) == m3scan.M3_E_ALIAS


@pytest_nodev
def test_slices_of_one_buffer():
    """Heads in each other's gaps are no overlap; one chunk more is."""
    token = 64 * 16
    s = (300 * token, token, 64)
    a = BWD.addr("q")
    d = attn_dims(q=s, k=s, v=s, dq=s, dk=s, dv=s)
    at = lambda h: a + h * 64 * 2
    assert BWD(dims=d, k=at(8), v=at(10)) == NODEVICE
    assert BWD(dims=d, dq=at(8)) == NODEVICE                                       # 8 heads behind q's
    assert BWD(dims=d, dq=at(8) - 16) == m3scan.M3_E_ALIAS
    assert BWD(dims=d, dq=at(8) + 16) == m3scan.M3_E_ALIAS                         # into q's next token
    b = BWD.addr("dq")
    assert BWD(dims=d, dk=b + 8 * 128, dv=b + 10 * 128) == NODEVICE
    assert BWD(dims=d, dk=b + 8 * 128, dv=b + 9 * 128) == m3scan.M3_E_ALIAS
    d.dv = (300 * (token + 8), token + 8, 64)
    assert BWD(dims=d, dk=b + 8 * 128, dv=b + 10 * 128) == m3scan.M3_E_ALIAS       # other distances cross
    # [b, 3, H, L, D]
    plane = 8 * 300 * 64
    s = (3 * plane, 64, 300 * 64)
    d = attn_dims(kv_heads=8, dq=s, dk=s, dv=s)
    assert BWD(cu=0, dims=d, dk=b + plane * 2, dv=b + 2 * plane * 2) == NODEVICE
    assert BWD(cu=0, dims=d, dk=b + plane * 2, dv=b + 2 * plane * 2 - 16) == m3scan.M3_E_ALIAS
    # keys and values of a page side by side
    half = 2 * 16 * 64
    s = (2 * half, 64, 16 * 64)
    d = cache_dims(seqlen=20, rotary_dim=32, k_cache=s, v_cache=s)
    c = APP.addr("k_cache")
    assert APP(dims=d, v_cache=c + half * 2) == NODEVICE
    assert APP(dims=d, v_cache=c + half * 2 - 16) == m3scan.M3_E_ALIAS


def test_workspaces():
    lib = m3attn.load()
    d = attn_dims()
    need = lib.m3_attention_backward_workspace_bytes(ctypes.byref(d), 0)
    part = 2 * 600 * 2 * 64 * 4                             # dk and dv of one part of the heads of a group
    assert need > 600 * 8 * 4 and (need - 600 * 8 * 4) % part == 0
    alone = attn_dims(kv_heads=8)                           # nothing to split
    assert lib.m3_attention_backward_workspace_bytes(ctypes.byref(alone), 0) == 600 * 8 * 4
    assert lib.m3_attention_backward_workspace_bytes(ctypes.byref(alone), 1) == 300 * 8 * 4
    assert lib.m3_attention_backward_workspace_bytes(ctypes.byref(attn_dims(head_dim=7)), 0) == 0
    assert BWD(cu=0, ws_bytes=need - 1) == m3scan.M3_E_WORKSPACE
    assert BWD(cu=0, workspace=0) == m3scan.M3_E_WORKSPACE
    d = cache_dims()
    need = lib.m3_attention_step_workspace_bytes(ctypes.byref(d))
    assert need > 0 and need % (8 * (2 + 64) * 4) == 0
    assert STEP(ws_bytes=need - 1) == m3scan.M3_E_WORKSPACE
    short = cache_dims(table_width=8)       # 128 positions: never cut
    assert lib.m3_attention_step_workspace_bytes(ctypes.byref(short)) == 0
    assert lib.m3_attention_step_workspace_bytes(ctypes.byref(cache_dims(flags=1))) == 0


@pytest_nodev
def test_step_needs_no_workspace_for_short_tables():
    assert STEP(dims=cache_dims(table_width=8), workspace=0, ws_bytes=0) == NODEVICE


def test_cache_sizes():
    for call in (APP, STEP):
        for field, value in [("page_size", 0), ("page_size", 1 << 31), ("num_pages", -1), ("num_pages", 1 << 31),
                             ("table_width", -1), ("table_width", 1 << 31)]:
            assert call(dims=call.make(**{field: value})) == m3scan.M3_E_DIMS, field
    for bad in (-8, 4, 12, 72):
        assert APP(dims=APP.make(rotary_dim=bad)) == m3scan.M3_E_DIMS and "rotary_dim" in m3scan.last_error()
    assert STEP(dims=cache_dims(seqlen=2)) == m3scan.M3_E_DIMS and "seqlen" in m3scan.last_error()
    assert STEP(dims=cache_dims(flags=1)) == m3scan.M3_E_DIMS
    assert APP(dims=APP.make(seqlen=1 << 24)) == m3scan.M3_E_DIMS
    assert FWD(dims=attn_dims(seqlen=1 << 30, heads=1024, kv_heads=1, q=(0, 0, 64), o=(0, 0, 64))) == m3scan.M3_E_DIMS


@pytest_nodev
def test_empty_sizes():
    assert FWD(dims=attn_dims(batch=0), q=0, k=0, v=0, o=0, cu=0) == NODEVICE
    assert FWD(dims=attn_dims(seqlen=0), q=0, k=0, v=0, o=0) == NODEVICE
    assert APP(dims=APP.make(seqlen=0), q=0, k=0, v=0, q_out=0, k_out=0) == NODEVICE
    assert APP(dims=APP.make(num_pages=0), k_cache=0, v_cache=0) == NODEVICE
    assert STEP(dims=cache_dims(batch=0), q=0, o=0, lens=0, page_table=0, workspace=0, ws_bytes=0) == NODEVICE
    assert STEP(dims=cache_dims(num_pages=0), k_cache=0, v_cache=0) == NODEVICE


def test_binding_refusals():
    """What the binding checks itself, with tensors on the CPU (which it refuses last)."""
    q, k = torch.zeros(2, 5, 4, 64), torch.zeros(2, 5, 2, 64)
    with pytest.raises(ValueError, match="GPU"):
        m3attn.m3_attention(q, k, k)
    with pytest.raises(ValueError, match="q must be"):
        m3attn.m3_attention(q[0], k[0], k[0])
    with pytest.raises(ValueError, match="v has shape"):
        m3attn.m3_attention(q, k, k[:, :4])
    with pytest.raises(ValueError, match="v has dtype"):
        m3attn.m3_attention(q, k, k.bfloat16())
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        m3attn.m3_attention(q.half(), k.half(), k.half())
    with pytest.raises(ValueError, match="dense"):
        m3attn.m3_attention(q, torch.zeros(2, 5, 2, 128)[..., ::2], k)
    with pytest.raises(ValueError, match="strides of 0"):
        m3attn.m3_attention(q, torch.zeros(64).expand(2, 5, 2, 64), k)
    with pytest.raises(ValueError, match="scale"):
        m3attn.m3_attention(q, k, k, scale=0.0)
    with pytest.raises(ValueError, match="cu_seqlens"):
        m3attn.m3_attention(q[0], k[0], k[0], torch.tensor([0, 5]))
    with pytest.raises(ValueError, match="lse is required"):
        m3attn.m3_attention_backward(q, k, k, q, None, q)
    with pytest.raises(ValueError, match="lse has shape"):
        m3attn.m3_attention_backward(q, k, k, q, torch.zeros(2, 5, 4), q)
    cache, table = torch.zeros(9, 2, 16, 64), torch.zeros(2, 4, dtype=torch.int32)
    lens = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="go together"):
        m3attn.m3_cache_append(k, k, cache, None, table, lens)
    with pytest.raises(ValueError, match="go together"):
        m3attn.m3_cache_append(k, None, cache, cache, table, lens)
    with pytest.raises(ValueError, match="k_cache has shape"):
        m3attn.m3_cache_append(k, k, cache[:, :1], cache, table, lens)
    with pytest.raises(ValueError, match="page_table has dtype"):
        m3attn.m3_cache_append(k, k, cache, cache, table.long(), lens)
    with pytest.raises(ValueError, match="page_table"):
        m3attn.m3_cache_append(k, k, cache, cache, table[0], lens)
    with pytest.raises(ValueError, match="lens has shape"):
        m3attn.m3_cache_append(k, k, cache, cache, table, lens[:1])
    with pytest.raises(ValueError, match="without q"):
        m3attn.m3_cache_append(k, k, cache, cache, table, lens, q_out=q)
    with pytest.raises(ValueError, match="GPU"):
        m3attn.m3_cache_append(k, k, cache, cache, table, lens, q=q)
    with pytest.raises(ValueError, match="q must be"):
        m3attn.m3_attention_step(q, cache, cache, table, lens)
    with pytest.raises(ValueError, match="lens is required"):
        m3attn.m3_attention_step(q[:, 0], cache, cache, table, None)
    with pytest.raises(ValueError, match="page_table has shape"):
        m3attn.m3_attention_step(q[:, 0], cache, cache, table[:1], lens)
    with pytest.raises(ValueError, match="GPU"):
        m3attn.m3_attention_step(q[:, 0], cache, cache, table, lens)


def test_table_sizes():
    """A page table of more bytes than 64 bits count is refused before its size is made."""
    for batch, width in [((1 << 31) - 1, (1 << 31) - 1), ((1 << 31) - 1, 1 << 30), (1 << 20, (1 << 31) - 1)]:
        assert APP(dims=APP.make(batch=batch, seqlen=0, table_width=width)) == m3scan.M3_E_DIMS, (batch, width)
        assert "page_table" in m3scan.last_error()
        assert STEP(dims=cache_dims(batch=batch, table_width=width)) == m3scan.M3_E_DIMS


@pytest.mark.parametrize("io", [m3attn.M3_BF16, m3attn.M3_F32])
@pytest.mark.parametrize("group", [2, 3, 5, 7, 10, 13, 64, 71, 1000, 1009])
@pytest.mark.parametrize("kv_heads,seqlen", [(1, 128), (1, 1024), (1, 16384), (1, 65536), (4, 16384), (8, 2048), (3, 40000)])
def test_parts_of_a_group_are_bounded(io, group, kv_heads, seqlen):
    """dk and dv in parts: at most about twice as many blocks as the GPU takes (1024; few ones 128), whatever the group
    divides into, and enough of them."""
    d = attn_dims(batch=1, seqlen=seqlen, heads=kv_heads * group, kv_heads=kv_heads, head_dim=128, io=io)
    need = m3attn.load().m3_attention_backward_workspace_bytes(ctypes.byref(d), 0)
    parts = need - seqlen * kv_heads * group * 4
    one = 2 * seqlen * kv_heads * 128 * 4
    assert parts % one == 0 and parts != one
    splits, blocks = max(1, parts // one), (seqlen + 127) // 128 * kv_heads
    assert splits <= group
    assert splits == 1 or blocks * splits <= 2 * 1024
    if io == m3attn.M3_BF16 and blocks > 256:
        assert splits == group or blocks * splits >= 1024


def test_scales_out_of_range():
    """Scales that fp32 does not hold: the binding's float would become 0, which stands for the default, and the library's
    product with log2 e infinite."""
    q, k = torch.zeros(2, 5, 4, 64), torch.zeros(2, 5, 2, 64)
    cache, table, lens = torch.zeros(9, 2, 16, 64), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad in (1e-50, 2.0 ** -150, -1e-50, float("nan")):
        with pytest.raises(ValueError, match="scale"):
            m3attn.m3_attention(q, k, k, scale=bad)
        with pytest.raises(ValueError, match="scale"):
            m3attn.m3_attention_backward(q, k, k, q, torch.zeros(2, 4, 5), q, scale=bad)
        with pytest.raises(ValueError, match="scale"):
            m3attn.m3_attention_step(q[:, 0], cache, cache, table, lens, scale=bad)
    for call in (FWD, BWD, STEP):
        for bad in (2.4e38, 3.4e38):
            assert call(dims=call.make(scale=bad)) == m3scan.M3_E_DIMS and "scale" in m3scan.last_error()


@pytest_nodev
def test_scales_at_the_ends_of_the_range():
    for call in (FWD, BWD, STEP):
        for scale in (2.0 ** -149, 1e-38, 2.3e38):
            assert call(dims=call.make(scale=scale)) == NODEVICE
