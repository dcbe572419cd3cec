"""Source checks of the 8-bit cache kernels' hand-written LDS reads (CPU only).

The compiler counts neither loads that go from memory to LDS nor what inline
assembly reads: a block that reads LDS waits for its own reads before it ends,
its outputs take no input's register, and where loads to LDS are read back a
wait for them comes first.
"""

import os
import re

import pytest

from block_wise_int4_amd import build as B


def _source(name):
    return open(os.path.join(B.CSRC, name)).read()


def _blocks(text):
    """(instructions, operands) of every inline asm statement with instructions."""
    found = re.findall(r'asm volatile\(\s*((?:"[^"]*"\s*)+)((?:[^;"]|"[^"]*")*);', text)
    return [("".join(re.findall(r'"([^"]*)"', code)), rest) for code, rest in found if "ds_read" in code]


def test_reads_of_tiles_wait_for_themselves():
    blocks = _blocks(_source("mnb_attn8_tiles.h"))
    assert len(blocks) == 3
    for code, operands in blocks:
        assert code.rstrip().endswith("s_waitcnt lgkmcnt(0)"), code
        outputs = operands.split(":")[1]
        assert outputs.count('"=') == outputs.count('"=&v"') == code.count("ds_read"), outputs
        if "ds_read_b128" in code:      # keys: loads to LDS have come back first
            assert code.startswith("s_waitcnt vmcnt("), code


@pytest.mark.parametrize("source", ["mnb_attn8.hip", "mnb_attn8_few.hip"])
def test_values_are_waited_for_before_they_are_read(source):
    text = _source(source)
    reads = [m.start() for m in re.finditer(r"read_values<", text)]
    waits = [m.start() for m in re.finditer(r"wait_loads<[^0]", text)]
    requests = [m.start() for m in re.finditer(r"request_values\(\);", text)]
    assert reads and waits
    for at in reads:        # a wait stands between the read and the request written before it
        before = [w for w in waits if w < at]
        assert before and not [r for r in requests if before[-1] < r < at]
    # the last tiles' loads have arrived before their place is used again
    assert re.search(r"wait_loads<0>\(\);\s*__syncthreads\(\);", text)


def test_queries_of_many_rows_are_waited_for():
    text = _source("mnb_attn8_rows.hip")
    load, wait = text.index("__builtin_amdgcn_global_load_lds"), text.index("s_waitcnt vmcnt(0)")
    assert load < wait < text.index("in_rows(col, 2 * j + half)")
