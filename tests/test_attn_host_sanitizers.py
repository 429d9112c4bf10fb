"""The host code of the attention operators (attn_api.hip) under AddressSanitizer and UndefinedBehaviorSanitizer, as
tests/test_block_host_sanitizers.py does for block_api.hip: the C-ABI files are compiled with the sanitizers on their host
pass only and linked with the regular build's kernels, and a child process runs tests/test_attn_host.py against that
library."""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

from state_space_sequence_m3_amd import build as m3build
from test_host_sanitizers import CSRC, OBJS, ROCM, ROOT, _runtime

CHILD = r"""
import sys
sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
from state_space_sequence_m3_amd import m3attn, m3scan
m3scan.load({lib!r})
assert m3attn.load()._name == {lib!r}
import pytest
sys.exit(pytest.main([{host!r}, "-q", "-p", "no:cacheprovider", "-k", "not structures and not index_maps"]))
"""


def test_attn_host_code_under_asan_and_ubsan(tmp_path):
    hipcc = os.path.join(ROCM, "bin", "hipcc")
    rt = _runtime()
    if not os.path.exists(hipcc) or rt is None:
        pytest.skip("hipcc or the clang sanitizer runtime is not installed")
    checked = ("api.hip", "block_api.hip", "attn_api.hip")
    others = [os.path.join(OBJS, s + ".o") for s in m3build.SOURCES if s not in checked]
    if not all(os.path.exists(o) for o in others):
        pytest.skip("the regular build's objects are missing (run the build first)")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]

    def compile_one(src):
        obj = str(tmp_path / (src + ".o"))
        cc = [hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
              "-I", os.path.join(ROOT, "include"), "-I", CSRC] + san + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cc, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-4000:]
        return obj

    with ThreadPoolExecutor(max_workers=3) as ex:
        objs = list(ex.map(compile_one, checked))
    lib = str(tmp_path / "libm3scan_san.so")
    ld = [hipcc, "--offload-arch=gfx950", "-shared", "-fPIC", "-fsanitize=address,undefined", "-shared-libasan",
          "-o", lib] + objs + others
    r = subprocess.run(ld, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ)
    env["LD_PRELOAD"] = rt
    env["ASAN_OPTIONS"] = "detect_leaks=0:halt_on_error=1:abort_on_error=1"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    code = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"), lib=lib,
                        host=os.path.join(ROOT, "tests", "test_attn_host.py"))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=600)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-6000:]
    assert r.returncode == 0, out[-6000:]
    assert " passed" in r.stdout, out[-3000:]
