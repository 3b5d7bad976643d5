"""A wait that runs out ends a kernel in order only if a warp's lanes leave it
together: the votes, shuffles and tcgen05 instructions behind it count on all of
them.  Read from the serving kernels' source: each wait is a whole warp's with one
answer, a single thread's, or one whose answer nobody takes."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "dynamic_hierarchical_sparse_b200", "csrc")


def _lines(name):
    text = open(os.path.join(CSRC, name)).read()
    return [re.sub(r"//.*", "", line) for line in text.split("\n")]


def _branch(lines, at):
    """The conditions of the blocks around a line, innermost first."""
    out, depth = [], 0
    for line in reversed(lines[:at]):
        depth += line.count("}") - line.count("{")
        if depth < 0:
            out.append(line.strip())
            depth = 0
    return out


@pytest.mark.parametrize("name", ["paged_attention.cu", "paged_prefix.cu"])
def test_waits(name):
    lines = _lines(name)
    warp = 0
    for i, line in enumerate(lines):
        if re.search(r"\bmbar_wait_warp\b", line):
            warp += 1
            assert not any("lane == 0" in c for c in _branch(lines, i)), line
        if re.search(r"\bmbar_wait(?:_spin)?(?:<\w+>)?\(", line):
            lone = any("lane == 0" in c for c in _branch(lines, i))
            dropped = "&never" in line
            assert lone or dropped, (i + 1, line)
    assert warp >= 3


@pytest.mark.parametrize("name", ["paged_attention.cu", "paged_prefix.cu"])
def test_no_wait_goes_by_an_earlier_calls_report(name):
    """The status word of these calls is not cleared by them, so no wait may end by what it says."""
    for line in _lines(name):
        for wait in re.findall(r"\bmbar_wait\w*(?:<\w+>)?\(", line):
            assert wait.endswith("<false>("), line
    text = open(os.path.join(CSRC, "common.cuh")).read()
    reads = re.findall(r"if \((.*)reinterpret_cast<volatile uint32_t\*>\(status\)", text)
    assert len(reads) == 2 and all(r.startswith("kHeed && ") for r in reads)


def test_the_warp_wait_votes():
    text = open(os.path.join(CSRC, "common.cuh")).read()
    body = text[text.index("bool mbar_wait_warp("):]
    assert re.search(r"return __all_sync\(0xffffffffu, mbar_wait\b", body[:body.index("\n}")])
