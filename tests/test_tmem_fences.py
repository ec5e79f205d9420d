"""Reading of the kernels' sources (no GPU): MMAs are ordered behind the wait
that lets them run.

A warp that has waited on an mbarrier for tensor memory (or for the operands
of an MMA) must execute tcgen05.fence::after_thread_sync before it issues
tcgen05 instructions that depend on that wait.  In every kernel, going back
from the block of code in which the elected lane issues MMAs, the fence comes
before any wait."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_block_self_b200", "csrc")


def _code(path):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


def _issuing_blocks(src):
    """(start, line) of every one-lane block that issues MMAs."""
    for m in re.finditer(r"if \((?:elect_one\(\)|lane == 0[^;{]*)\) \{", src):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(src[i], 0)
            i += 1
        if re.search(r"\bmma_(ss|ts)\(", src[m.end():i]):
            yield m.start(), src.count("\n", 0, m.start()) + 1


KERNELS = sorted(p for p in glob.glob(os.path.join(CSRC, "*.cu")) if list(_issuing_blocks(_code(p))))


def test_kernels_found():
    names = {os.path.basename(p) for p in KERNELS}
    assert {"attn_bwd_sm100a.cu", "block_bwd_sm100a.cu"} <= names


@pytest.mark.parametrize("path", KERNELS, ids=os.path.basename)
def test_mmas_are_fenced_behind_their_waits(path):
    src = _code(path)
    for at, line in _issuing_blocks(src):
        wait = max((m.start() for m in re.finditer(r"\bwait(_bar)?\(", src[:at])), default=-1)
        assert src.rfind("tc_fence_after()", 0, at) > wait, f"{os.path.basename(path)}: MMAs issued near line {line}"
