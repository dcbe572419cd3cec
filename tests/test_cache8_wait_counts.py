"""The counts of the 8-bit cache kernels' hand-written waits, in what the compiler made of
them (CPU only: the two kernels are compiled to assembly).

`s_waitcnt vmcnt(N)` in a kernel's inline assembly lets the last N loads still be under
way; which loads these are rests on the order and number that the compiler gives them. A
tile's key codes are read behind the first wait of the loop, its value codes behind the
second; both arrive in LDS by loads marked `lds`, those of the keys first.
"""

import os
import re
import subprocess

import pytest

from block_wise_int4_amd import build as B

LOAD = re.compile(r"(buffer|global|flat|scratch)_")


def _kernels(source, tmp_path):
    """(template arguments, lines) of every kernel of a source file."""
    out = os.path.join(tmp_path, source + ".s")
    subprocess.run([B.hipcc(), *B.HIPCC_FLAGS, "-I", os.path.join(B.ROOT, "include"), "-S", "--offload-device-only",
                    os.path.join(B.CSRC, source), "-o", out], check=True, capture_output=True)
    text = open(out).read()
    for m in re.finditer(r"^(_ZN3mnb\S*attn8_(?:few_)?kernel\S*):", text, re.M):
        yield m.group(1), [l.strip() for l in text[m.end(): text.index(".Lfunc_end", m.end())].splitlines()]


def _events(lines):
    """In program order: 'lds' (a load into LDS), 'load' (any other use of the
    counter), ('hand', N) (a wait of inline assembly), ('label', name),
    ('branch', name)."""
    hand = False
    for l in lines:
        if "#ASMSTART" in l or "#ASMEND" in l:
            hand = "#ASMSTART" in l
        elif LOAD.match(l):
            yield "lds" if l.endswith(" lds") else "load"
        elif hand and (m := re.match(r"s_waitcnt vmcnt\((\d+)\)", l)):
            yield "hand", int(m.group(1))
        elif m := re.match(r"(\.LBB\w+):", l):
            yield "label", m.group(1)
        elif m := re.match(r"s_c?branch\w*\s+(\.LBB\w+)", l):
            yield "branch", m.group(1)


def _check(name, lines):
    codes = 4 * int(re.search(r"Li(64|128)", name).group(1)) // 64    # loads of a tile's key or value codes
    events = list(_events(lines))
    # the loop: from its label to the branch back, with both tiles' loads in it
    place = {e[1]: i for i, e in enumerate(events) if e[0] == "label"}
    loops = [(place[e[1]], i) for i, e in enumerate(events) if e[0] == "branch" and place.get(e[1], i) < i]
    loops = [(i, j) for i, j in loops if events[i:j].count("lds") == 2 * codes]
    assert len({i for i, _ in loops}) == 1, name
    begin, end = loops[0]
    assert not {"lds", "load"} & {e for e in events[end: loops[-1][1]] if isinstance(e, str)}, name
    loop, before = events[begin:end], events[:begin]
    assert before.count("lds") == 2 * codes, name
    # no load in the loop is jumped over: forward branches skip none
    for i, e in enumerate(loop):
        if e[0] == "branch" and ("label", e[1]) in loop[i:]:
            skipped = loop[i: loop.index(("label", e[1]))]
            assert not {"lds", "load"} & {s for s in skipped if isinstance(s, str)}, name
    waits = [(i, e[1]) for i, e in enumerate(loop) if e[0] == "hand"]
    assert len(waits) == 2, (name, waits)
    (first, behind), (second, later) = waits
    tiles = [i for i, e in enumerate(loop) if e == "lds"]
    assert first < tiles[0] and tiles[codes - 1] < second < tiles[codes], name

    def loads(part):
        return sum(e in ("lds", "load") for e in part)
    # a wait is long enough if N loads or more were made since the last one it is for: of the tile before the
    # loop, and of the one a turn ago
    start = [i for i, e in enumerate(before) if e == "lds"]
    for since in (before[start[codes - 1] + 1:], loop[tiles[codes - 1] + 1:]):
        assert loads(since) + loads(loop[:first]) >= behind, f"{name}: keys"
    for since in (before[start[-1] + 1:], loop[tiles[-1] + 1:]):
        assert loads(since) + loads(loop[:second]) >= later, f"{name}: values"


@pytest.mark.parametrize("source,kernels", [("mnb_attn8.hip", 8), ("mnb_attn8_few.hip", 32)])
def test_waits_are_for_loads_that_came_before(source, kernels, tmp_path):
    found = list(_kernels(source, tmp_path))
    assert len(found) == kernels
    for name, lines in found:
        _check(name, lines)
