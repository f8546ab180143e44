"""The kernels' asynchronous copies, as the compiler sees them: every inline-assembly statement that starts,
groups or waits for copies to shared memory must say that it touches memory.  A thread that reads its own
copies behind its own wait, with no barrier in between, relies on that alone: a volatile statement
without it does not keep plain loads from moving across it."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_bwd_b200",
                    "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def statements(text):
    """The inline-assembly statements of a source, comments removed, each up to its closing parenthesis."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\basm\b[\s\w]*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield text[m.start():i]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_asynchronous_copies_are_memory_accesses_to_the_compiler(path):
    found = [s for s in statements(open(path).read()) if "cp.async" in s]
    for s in found:
        assert "volatile" in s and re.search(r':\s*"memory"\s*\)$', s), s
    if os.path.basename(path) == "real_common.cuh":
        assert len(found) >= 8  # the helpers that the kernels share
