"""Wait states around the hand-written LDS loads along every path: a memory
instruction may use a scalar register five wait states after a vector
instruction wrote it, and the compiler keeps that distance for its own
instructions only.  test_w8a8_listing.py reads the listing upwards as it
stands; here a label leads on to every branch that names it, so that the end of
a loop's body counts as what comes before its head."""
import os
import re
import subprocess

import pytest

from test_w8a8_listing import LOAD, WRITE
from weight_only_bit_rtn_amd import build

LABEL = re.compile(r"([\w.$]+):$")
BRANCH = re.compile(r"s_(?:c?branch\w*|call\w*) (?:\S+, )?([\w.$]+)$")
WITHOUT_NEXT = ("s_branch ", "s_endpgm", "s_setpc_b64 ")
STATES = 5


def instructions(listing: str) -> list[str]:
    """Instructions and labels, without comments and directives."""
    lines = [line.split(";")[0].strip() for line in listing.split("\n")]
    return [line for line in lines if line and (not line.startswith(".") or LABEL.match(line))]


def close_writes(listing: str) -> tuple[int, list[str]]:
    """(LDS loads seen, those whose descriptor was written too shortly before on some path)."""
    lines = instructions(listing)
    sources: dict[str, list[int]] = {}
    for i, line in enumerate(lines):
        branch = BRANCH.match(line)
        if branch:
            sources.setdefault(branch[1], []).append(i)
    loads, close = 0, []
    for i, line in enumerate(lines):
        load = LOAD.match(line)
        if not load:
            continue
        loads += 1
        first, last = int(load[1]), int(load[2])
        # (place, wait states between it and the load), the place's own instruction not yet looked at
        todo, seen = [(i, 0)], set()
        while todo:
            at, states = todo.pop()
            label = LABEL.match(lines[at]) if at != i else None
            before = list(sources.get(label[1], ())) if label else []
            if at > 0 and not lines[at - 1].startswith(WITHOUT_NEXT):
                before.append(at - 1)
            for j in before:
                if (j, states) in seen:
                    continue
                seen.add((j, states))
                write = WRITE.match(lines[j])
                if write and int(write[1]) <= last and int(write[2] or write[1]) >= first:
                    close.append(f"{lines[j]} | {line}")
                    continue
                nop = re.match(r"s_nop (\d+)", lines[j])
                then = states + (int(nop[1]) + 1 if nop else 0 if LABEL.match(lines[j]) else 1)
                if then < STATES:
                    todo.append((j, then))
    return loads, close


LOADED = "buffer_load_dwordx4 v1, s[8:11], 0 offen lds"


def test_a_write_before_the_load_is_found():
    assert close_writes(f"v_readfirstlane_b32 s9, v2\ns_mov_b32 m0, s3\ns_nop 0\n{LOADED}")[1]
    assert close_writes(f"v_readfirstlane_b32 s9, v2\ns_nop 3\ns_mov_b32 m0, s3\n{LOADED}") == (1, [])
    assert close_writes(f"v_readfirstlane_b32 s12, v2\n{LOADED}") == (1, [])


def test_a_write_at_the_end_of_a_loop_is_found():
    # the write lies below the load and reaches it by the branch back
    loop = f"s_nop 7\n.LBB0_1:\ns_mov_b32 m0, s3\ns_nop 0\n{LOADED}\ns_nop 7\n%s\ns_cbranch_scc1 .LBB0_1\ns_endpgm"
    assert close_writes(loop % "v_readlane_b32 s10, v3, 0")[1]
    assert close_writes(loop % "v_readlane_b32 s10, v3, 0\ns_nop 2") == (1, [])
    assert close_writes(loop % "v_readlane_b32 s12, v3, 0") == (1, [])


def test_what_an_unconditional_branch_leaves_behind_is_not_before():
    text = f"s_branch .LBB0_2\n.LBB0_1:\nv_readlane_b32 s10, v3, 0\ns_branch .LBB0_3\n.LBB0_2:\n{LOADED}\n.LBB0_3:\ns_endpgm"
    assert close_writes(text) == (1, [])
    assert close_writes(text.replace("s_branch .LBB0_3", "s_branch .LBB0_2"))[1]


@pytest.mark.parametrize("source", ["w8a8_gemm.hip", "w8a8_grad.hip", "w8a8_skinny.hip"])
def test_descriptors_are_settled_on_every_path(source, tmp_path):
    out = tmp_path / "listing.s"
    subprocess.run([build.HIPCC, *build.FLAGS, "--offload-device-only", "-S",
                    os.path.join(build.CSRC, source), "-o", str(out)], check=True,
                   stderr=subprocess.DEVNULL, timeout=600)
    loads, close = close_writes(out.read_text())
    assert loads > 0
    assert close == []
