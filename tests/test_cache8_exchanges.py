"""Source checks of what lanes of a wave hand one another through LDS without a workgroup
barrier (CPU only): a fence stands between the stores and the loads, and before the
place is used again. The compiler owes only one lane's order.
"""

import os

import pytest

from block_wise_int4_amd import build as B


def _in_order(name, marks):
    """Every mark stands in the source, once after the one before it."""
    text = open(os.path.join(B.CSRC, name)).read()
    at = 0
    for mark in marks:
        found = text.find(mark, at)
        assert found >= 0, f"{name}: no `{mark}` behind offset {at}"
        at = found + len(mark)


FENCE = "wave_fence();"


@pytest.mark.parametrize("name,marks", [
    # products by column, read by key; digits by key, read by column; the next tile's products
    ("mnb_attn8_few.hip", ["<i32x4 *>(s_products + col", FENCE, "s_products + 3 * i * kScoreStride + lane", FENCE,
                           "s_digits[(3 * i + t) * kDigitStride + lane] =", FENCE,
                           "(s_digits + (col < kColumns ? col : 0)", FENCE, "request_values();\n    }"]),
    # whole rows of results; pieces in two halves through one place
    ("mnb_attn8_rows.hip", ["<u32x2 *>(in_rows(col_now, 4 * d", FENCE, "<const u32x4 *>(in_rows(row, piece_now))",
                            "<f4 *>(in_rows(col_now, 8 * d", FENCE, "<const f4 *>(in_rows(row, piece_now))", FENCE]),
    # a token's cosines and sines
    ("mnb_rope.hip", ["s_turn[wave][i] = turn_of", FENCE, "s_turn[wave][unit[i]"]),
])
def test_a_fence_stands_between_lanes(name, marks):
    _in_order(name, marks)


def test_the_fence_keeps_all_memory_in_order():
    _in_order("mnb_device.h", ["void wave_fence() {", '__builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");',
                               "__builtin_amdgcn_wave_barrier();", "}"])
