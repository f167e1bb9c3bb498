"""Loops around warp-collective loads of the accumulators, read as source."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_nf4_quantized_blk_b200", "csrc")


def _loops(text):
    """(first line, body) of every braced for loop."""
    for m in re.finditer(r"\bfor \(", text):
        i, depth = m.end(), 1
        while depth:  # the header's closing parenthesis
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        i += len(text[i:]) - len(text[i:].lstrip())
        if text[i] != "{":
            continue
        start, depth = i, 0
        while True:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
            if depth == 0:
                break
        yield text.count("\n", 0, m.start()) + 1, text[start:i]


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh"))))
def test_no_lane_leaves_a_loop_of_collective_loads(name):
    """tcgen05.ld is executed by all lanes of a warp together: no lane may skip to the next iteration (`continue`)
    between one of a loop's loads and the next."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    bad = [line for line, body in _loops(text) if re.search(r"\btmem_ld_32x32b.*\bcontinue;", body, re.S)]
    assert not bad, bad
