"""What the attention backward kernel's source has to keep, and no run can show:
a warp that works is no proof that its lanes were together."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dit_long_sequence_gb300", "csrc")


@pytest.fixture(scope="module")
def kernel():
    with open(os.path.join(CSRC, "attn_bwd.cu"), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _block(text, start):
    """The braces' contents from the first one behind `start`."""
    at = text.index("{", text.index(start))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i]
    raise AssertionError("unbalanced braces")


def test_no_lane_leaves_the_loops_with_warp_wide_loads(kernel):
    """Loads of tensor memory are .aligned: all 32 lanes together.  A lane whose
    row is not there skips its stores, not the rest of an iteration, and the warp
    comes together before the next."""
    softmax = _block(kernel, "void soften(")
    assert "tmem_ld32(" in softmax and not re.search(r"\bcontinue\b", softmax)
    gradient = _block(softmax, "for (int cc = c0;")
    assert "tmem_ld32(" in gradient and gradient.rstrip().endswith("__syncwarp();")
