"""A bare barrier builtin waits for nothing: where it hands a stage of LDS back
to loads that write it, the source itself has to wait for the wave's reads of
that stage first (the compiler may place their waits after the barrier)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a4_rank_corrected_quantize_amd",
                    "csrc")


def test_bare_barriers_follow_a_wait_for_lds_reads():
    found = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.hip"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        statements = [s.strip() for s in text.split(";")]
        for before, s in zip(statements, statements[1:]):
            if s == "__builtin_amdgcn_s_barrier()":
                found += 1
                assert "s_waitcnt" in before and "lgkmcnt(0)" in before, (os.path.basename(path), before)
    assert found
