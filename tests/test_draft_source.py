"""The tensor-core attention kernels' sources, without a GPU: what a wait that has
run out decides for a warp, it decides for all of its lanes.

Another warp may raise the CTA's abort flag at any time, so lanes that read it on
their own may differ; those that leave would be missed in the next vote or shuffle
of the whole warp, which then need not end.  One elected thread may read it as it
likes, a warp through a vote."""
import os
import re

import pytest

from block_fp8_expert_gb300 import build as B


def _lone_reads(text):
    """Lines that read *dead outside of one elected thread's code."""
    found, opened, depth = [], [], 0
    for number, line in enumerate(text.split("\n"), 1):
        code = line.split("//")[0]
        alone = "elect_one()" in code
        if re.search(r"\*\s*dead\b(?!\s*=)", code) and not alone and not opened:
            found.append(number)
        before = depth
        depth += code.count("{") - code.count("}")
        while opened and depth <= opened[-1]:
            opened.pop()
        if alone and depth > before:
            opened.append(before)
    return found


@pytest.mark.parametrize("name", ["draft_attention.cu", "expanded_attention.cu"])
def test_the_abort_flag_decides_for_whole_warps(name):
    text = open(os.path.join(B.CSRC, name)).read()
    assert "dead" in text
    assert _lone_reads(text) == []


def test_a_lone_read_is_found():
    assert _lone_reads("for (;;) {\n  if (tc::elect_one()) {\n    if (*dead) break;\n  }\n  if (*dead) continue;\n}") == [5]
    assert _lone_reads("if (tc::elect_one() && !*dead) {\n  x();\n}\nvolatile int* const dead = &flag;") == []
