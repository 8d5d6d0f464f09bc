"""Host-side check of the inline PTX: an instruction that a whole warp must reach together (.aligned) is issued
by a wrapper that lets the warp's lanes meet first, so that no caller has to know where its lanes parted."""
from __future__ import annotations

import glob
import os
import re

import pytest

from dit_block_b200 import build


def functions_with(text: str, instruction: str):
    """The bodies of the functions whose inline PTX holds `instruction`, up to it."""
    text = re.sub(r"//[^\n]*", "", text)
    for at in (m.start() for m in re.finditer(re.escape(instruction), text)):
        start = text.rfind("\n{\n", 0, at)
        assert start >= 0, instruction
        yield text[start:at]


@pytest.mark.parametrize("instruction", [
    "tcgen05.ld.sync.aligned", "tcgen05.alloc.", "tcgen05.relinquish_alloc_permit.", "tcgen05.dealloc.",
    "barrier.cluster.arrive.release.aligned"])
def test_lanes_meet_before_a_warp_aligned_instruction(instruction):
    found = 0
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu")) + glob.glob(os.path.join(build.CSRC, "*.cuh"))):
        with open(path) as f:
            for body in functions_with(f.read(), instruction):
                found += 1
                assert "__syncwarp();" in body, f"{os.path.basename(path)}: {instruction} without __syncwarp() before it"
    assert found
