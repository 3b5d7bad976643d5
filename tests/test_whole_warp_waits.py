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
        if "paged_wait_warp(" in line:
            warp += 1
            assert not any("lane == 0" in c for c in _branch(lines, i)), line
        if re.search(r"\b(?:paged|mbar)_wait(?:_spin)?\(", line):
            lone = any("lane == 0" in c for c in _branch(lines, i))
            dropped = "&never" in line
            assert lone or dropped, (i + 1, line)
    assert warp >= 3


@pytest.mark.parametrize("name", ["paged_attention.cu", "paged_prefix.cu", "paged.cuh"])
def test_no_wait_goes_by_an_earlier_calls_report(name):
    """The status word of these calls is not cleared by them, so no wait may end by what it says: the waits that
    read it are given none."""
    waits = [line for line in _lines(name) if re.search(r"\bmbar_wait(?:_spin)?\(", line)]
    for line in waits:
        assert "&never, nullptr" in line or "abort_flag, nullptr)" in line, line
    assert len(waits) >= 1


def test_a_wait_that_ran_out_is_reported_at_the_end():
    """Each kernel with waits looks at its CTA's abort flag behind the last of them."""
    for name, kernels in (("paged_attention.cu", 2), ("paged_prefix.cu", 1)):
        text = open(os.path.join(CSRC, name)).read()
        ends = [text[m.start():] for m in re.finditer(r"^__global__ .*\n(?:.*\n)?.*paged_(?:mma|f32|prefix)_kernel\(", text, re.M)]
        assert len(ends) == kernels
        for body in ends:
            body = body[:body.index("\n}\n")]
            assert "report_abort(" in body and "wait(" not in body[body.index("report_abort("):]


def test_the_warp_wait_votes():
    text = open(os.path.join(CSRC, "paged.cuh")).read()
    body = text[text.index("bool paged_wait_warp("):]
    assert re.search(r"return __all_sync\(0xffffffffu, paged_wait\(", body[:body.index("\n}")])
