"""The host code of the 8-bit activation entry points (abi_w8a8.hip: argument
checks, workspace sizes, status codes) under AddressSanitizer and
UndefinedBehaviorSanitizer, host code only: rebuilt with them, linked with the
library's other objects, and put through every refusal of test_w8a8_host in a
child process.  Nothing runs on a GPU."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

from test_sanitizers import SAN_ENV, _clang_asan_runtime, _sanitizer_report

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

CHILD = """
import sys
sys.path[:0] = [%r, %r]
import weight_only_bit_rtn_amd as lw
lw.load_library(sys.argv[1])
import test_w8a8_host as t
wrong = [(f.__name__, a, s, f(lw, **a)) for f, a, s in t.REFUSED if f(lw, **a) != s]
for f in t.ALL:
    assert f(lw, T=0) == 0
for T in (1, 3, 64, 65, 4096, 1 << 20):
    for N in (1, 63, 4096, 1 << 15):
        for K in (32, 4096, 65536):
            assert lw.linear_w8a8_workspace_bytes(T, N, K, 0) >= 0 and lw.gated_w8a8_workspace_bytes(T, N, K, 2) >= 0
            assert lw.linear_w8a8_grad_workspace_bytes(T, N, K) > 0 and lw.gated_w8a8_grad_workspace_bytes(T, N, K) > 0
print("refusals:", len(t.REFUSED), "wrong:", wrong)
sys.exit(1 if wrong else 0)
"""


def test_refusals_under_sanitizers(tmp_path):
    from weight_only_bit_rtn_amd import build as lib_build
    rt = _clang_asan_runtime()
    if rt is None:
        pytest.skip("no clang AddressSanitizer runtime in this ROCm install")
    objs = []
    for src in lib_build.SOURCES:
        obj = os.path.join(lib_build._obj_dir(), os.path.splitext(src)[0] + ".o")
        if not os.path.exists(obj):
            obj = lib_build._compile(src)
        objs.append(obj)
    san_obj = str(tmp_path / "abi_w8a8_san.o")
    host_san = []
    for flag in ("-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all"):
        host_san += ["-Xarch_host", flag]
    r = subprocess.run([lib_build.HIPCC, *lib_build.FLAGS, *host_san, "-c",
                        os.path.join(lib_build.CSRC, "abi_w8a8.hip"), "-o", san_obj], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    objs = [san_obj if o.endswith(os.sep + "abi_w8a8.o") else o for o in objs]
    so = str(tmp_path / "liblowbit_w8a8_san.so")
    r = subprocess.run([lib_build.HIPCC, f"--offload-arch={lib_build.ARCH}", "-shared", "-fPIC", "-o", so, *objs, rt],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, LD_PRELOAD=rt, **SAN_ENV)
    r = subprocess.run([sys.executable, "-c", CHILD % (ROOT, HERE), so], capture_output=True, text=True, env=env,
                       timeout=600)
    assert not _sanitizer_report(r), r.stderr[-4000:]
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
