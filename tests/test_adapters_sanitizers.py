"""The host code of the adapters' and the AdamW step's entry points (abi_lora.hip,
abi_adamw.hip: argument checks, workspace sizes) under AddressSanitizer and
UndefinedBehaviorSanitizer, host code only: rebuilt with them, linked with the library's other
objects, and put through every refusal of test_adapters_host in a child process.  Nothing runs
on a GPU."""
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
import test_adapters_host as t
wrong = [(f.__name__, a, s, f(lw, **a)) for f, a, s in t.REFUSED if f(lw, **a) != s]
wrong += [(f.__name__, a) for f, a in t.EMPTY if f(lw, **a) != 0]
for s in t.SIZES:
    assert lw.lora_workspace_bytes(*s) > 0 and lw.lora_grad_workspace_bytes(*s) > 0
print("refusals:", len(t.REFUSED), "wrong:", wrong)
sys.exit(1 if wrong else 0)
"""


def test_refusals_under_sanitizers(tmp_path):
    from weight_only_bit_rtn_amd import build as lib_build
    rt = _clang_asan_runtime()
    if rt is None:
        pytest.skip("no clang AddressSanitizer runtime in this ROCm install")
    host_san = []
    for flag in ("-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all"):
        host_san += ["-Xarch_host", flag]
    objs = []
    for src in lib_build.SOURCES:
        name = os.path.splitext(src)[0]
        obj = os.path.join(lib_build._obj_dir(), name + ".o")
        if name in ("abi_lora", "abi_adamw"):
            obj = str(tmp_path / (name + "_san.o"))
            r = subprocess.run([lib_build.HIPCC, *lib_build.FLAGS, *host_san, "-c", os.path.join(lib_build.CSRC, src),
                                "-o", obj], capture_output=True, text=True)
            assert r.returncode == 0, r.stderr[-4000:]
        elif not os.path.exists(obj):
            obj = lib_build._compile(src)
        objs.append(obj)
    so = str(tmp_path / "liblowbit_adapters_san.so")
    r = subprocess.run([lib_build.HIPCC, f"--offload-arch={lib_build.ARCH}", "-shared", "-fPIC", "-o", so, *objs, rt],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, LD_PRELOAD=rt, **SAN_ENV)
    r = subprocess.run([sys.executable, "-c", CHILD % (ROOT, HERE), so], capture_output=True, text=True, env=env,
                       timeout=600)
    assert not _sanitizer_report(r), r.stderr[-4000:]
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
