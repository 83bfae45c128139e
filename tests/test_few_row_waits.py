"""Loads that go to LDS by inline assembly are unknown to the compiler, which so
leaves them out of the waits that it puts before a barrier.  In the few-row
linear's forms with X in the ring, every load has to be home at the barriers
behind the loop over the stages, on every path to them: also on that of a wave
that has no stage of its own (rows of less than 256 channels per wave), whose
loads are operands of the epilogue that the other waves read.  No GPU: the walk is
over the assembly that the compiler makes of the source."""
import os
import re
import shutil
import subprocess

import pytest

from w4a4_rank_corrected_quantize_amd import build as B

CONDITIONAL, LABEL = re.compile(r"s_cbranch_\w+\s+(\S+)"), re.compile(r"(\.L\w+):")


def _kernels(text):
    """Name and instructions of every kernel: (labels, [(instruction, inside inline assembly)])."""
    name = None
    for line in text.splitlines():
        head = re.match(r"(_ZN\w+):", line)
        if head:
            name, labels, code, inline = head.group(1), {}, [], False
            continue
        if name is None:
            continue
        if line.startswith(".Lfunc_end"):
            yield name, labels, code
            name = None
            continue
        if "#ASMSTART" in line or "#ASMEND" in line:
            inline = "#ASMSTART" in line
            continue
        at = LABEL.match(line)
        if at:
            labels[at.group(1)] = len(code)
            continue
        line = line.split(";")[0].strip()
        if line and not line.startswith("."):
            code.append((line, inline))


def _barriers_with_loads_under_way(labels, code):
    """Compiler-made barriers of a kernel, and those that a path reaches with a load to LDS under way."""
    seen, todo, bad = set(), [(0, False)], set()
    while todo:
        at, loads = todo.pop()
        while at < len(code) and (at, loads) not in seen:
            seen.add((at, loads))
            line, inline = code[at]
            at += 1
            if "load_lds" in line:
                loads = True
            elif line.startswith("s_waitcnt") and "vmcnt(0)" in line:
                loads = False
            elif line == "s_barrier" and not inline and loads:
                bad.add(at - 1)
            elif line.startswith("s_endpgm"):
                break
            elif line.startswith("s_branch"):
                at = labels[line.split()[1]]
            elif CONDITIONAL.match(line):
                todo.append((labels[CONDITIONAL.match(line).group(1)], loads))
    return sum(1 for line, inline in code if line == "s_barrier" and not inline), bad


def test_the_walk_finds_a_path_without_a_wait():
    """The walk itself, on a loop that a wave may pass by."""
    load, wait = ("global_load_lds_dwordx4 v1, s[2:3]", True), ("s_waitcnt vmcnt(0)", True)
    body = [load, ("s_cbranch_scc1 .Lend", False), wait, ("s_branch .Lend", False)]
    assert _barriers_with_loads_under_way({".Lend": 4}, body + [("s_barrier", False), ("s_endpgm", False)]) == (1, {4})
    assert _barriers_with_loads_under_way({".Lend": 4}, body + [wait, ("s_barrier", False), ("s_endpgm", False)]) == (1, set())


def test_no_epilogue_operand_is_under_way_at_the_sums(tmp_path):
    if not os.path.exists(B.HIPCC) and shutil.which("hipcc") is None:
        pytest.skip("no hipcc")
    out = str(tmp_path / "few.s")
    subprocess.run([B.HIPCC] + B.COMMON + B.SOURCES["w4a4_few.hip"] + ["--offload-device-only", "-S",
                   os.path.join(B.CSRC, "w4a4_few.hip"), "-o", out], check=True, capture_output=True)
    with open(out) as f:
        text = f.read()
    forms = 0
    for name, labels, code in _kernels(text):
        # w4a4_few_kernel<FORM, RT, CT, GATED, WN, WK, DEPTH, XB = 0, XW>
        if not re.search(r"w4a4_few_kernelI(?:L\w\d+E){3}Lb\dE(?:Li\d+E){3}Li0ELb\dEE", name):
            continue
        forms += 1
        barriers, bad = _barriers_with_loads_under_way(labels, code)
        assert barriers >= 2 and not bad, (name, barriers, sorted(bad))
    assert forms >= 24
