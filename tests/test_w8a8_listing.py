"""Wait states around the hand-written LDS loads, read from the compiler's own
listing of the kernels: a memory instruction may use a scalar register five wait
states after a vector instruction wrote it, and the compiler keeps that distance
for its own instructions only.  Straight-line distance, which is what there is:
a label in between ends the search, the branch to it being a state of its own."""
import os
import re
import subprocess

import pytest

from weight_only_bit_rtn_amd import build

LOAD = re.compile(r"buffer_load_dwordx4 v\d+, s\[(\d+):(\d+)\], 0 offen lds")
WRITE = re.compile(r"v_\w+ s\[?(\d+)(?::(\d+))?")


def close_writes(listing: str) -> tuple[int, list[str]]:
    """(LDS loads seen, those whose descriptor was written too shortly before)."""
    lines = [line.split(";")[0].strip() for line in listing.split("\n")]
    lines = [line for line in lines if line and not line.startswith(".")]
    loads, close = 0, []
    for i, line in enumerate(lines):
        load = LOAD.match(line)
        if not load:
            continue
        loads += 1
        first, last = int(load[1]), int(load[2])
        states, j = 0, i - 1
        while states < 5 and j >= 0:
            write = WRITE.match(lines[j])
            if write and int(write[1]) <= last and int(write[2] or write[1]) >= first:
                close.append(f"{lines[j]} | {line}")
                break
            nop = re.match(r"s_nop (\d+)", lines[j])
            states += int(nop[1]) + 1 if nop else 0 if lines[j].endswith(":") else 1
            j -= 1
    return loads, close


def test_close_writes_are_found():
    load = "buffer_load_dwordx4 v1, s[8:11], 0 offen lds"
    assert close_writes(f"v_readfirstlane_b32 s9, v2\ns_mov_b32 m0, s3\ns_nop 0\n{load}")[1]
    assert close_writes(f"v_readlane_b32 s11, v2, 3\ns_mov_b32 m0, s3\ns_nop 0\n{load}")[1]
    assert not close_writes(f"v_readfirstlane_b32 s12, v2\ns_nop 0\n{load}")[1]
    assert close_writes(f"v_readfirstlane_b32 s9, v2\ns_nop 3\ns_mov_b32 m0, s3\n{load}") == (1, [])


@pytest.mark.parametrize("source", ["w8a8_gemm.hip", "w8a8_grad.hip", "w8a8_skinny.hip"])
def test_descriptors_are_settled(source, tmp_path):
    out = tmp_path / "listing.s"
    subprocess.run([build.HIPCC, *build.FLAGS, "--offload-device-only", "-S",
                    os.path.join(build.CSRC, source), "-o", str(out)], check=True,
                   stderr=subprocess.DEVNULL, timeout=600)
    loads, close = close_writes(out.read_text())
    assert loads > 0
    assert close == []
