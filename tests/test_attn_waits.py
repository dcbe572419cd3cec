"""Source checks of the attention kernels' hand-written barriers (CPU only).

Loads that go from memory to LDS are written without the compiler's counting:
where waves share the tiles, a barrier before the next loads has to wait both
for the wave's own loads (vmcnt) and for its own LDS reads (lgkmcnt), or
another wave's load could overwrite a tile that is still being read.
"""

import os
import re

import pytest

from block_wise_int4_amd import build as B


def _barriers(source):
    """The text of every inline asm statement that holds a barrier."""
    text = open(os.path.join(B.CSRC, source)).read()
    return [a for a in re.findall(r'asm volatile\(\s*((?:"[^"]*"\s*)+)', text) if "s_barrier" in a]


def test_cross_kernel_has_hand_written_barriers():
    assert _barriers("mnb_cross.hip")


@pytest.mark.parametrize("source", ["mnb_attn.hip", "mnb_cross.hip", "mnb_kv.hip"])
def test_barriers_wait_for_loads_to_lds_and_for_lds_reads(source):
    for asm in _barriers(source):
        wait = asm[: asm.index("s_barrier")]
        assert "vmcnt(0)" in wait and "lgkmcnt(0)" in wait, asm
