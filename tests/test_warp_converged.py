"""Accesses to tensor memory are a whole warp's: where lanes have gone different ways before one, they meet again first. And
what one warp's MMAs wrote is read by another's lanes only behind a barrier between the two fences for it. Read from the
source: what a run does where this is missing is up to the compiler."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_fa2_attn_gb300", "csrc")
WHOLE_WARP = r"tmem_(?:ld|st)(?:8|16|32|_wait)\("


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def _body(code, at):
    """The block that begins at the first open brace from `at` on."""
    start = code.index("{", at)
    depth = 0
    for i in range(start, len(code)):
        depth += {"{": 1, "}": -1}.get(code[i], 0)
        if depth == 0:
            return code[start + 1:i], i + 1
    raise AssertionError("no end")


@pytest.mark.parametrize("name", ["prefix.cu", "tree.cu"])
def test_stores_of_some_lanes_between_loads_of_all(name):
    # loops over columns that load from tensor memory and store the rows that a warp's lanes have
    code = _code(name)
    seen = 0
    for m in re.finditer(r"for \(int cc = ", code):
        body, _ = _body(code, m.end())
        if "pack_bf16x2" not in body or not re.search(r"tmem_ld(?:8|32)\(", body):
            continue
        seen += 1
        after = body[body.rindex("tmem_ld_wait();"):]
        assert not re.search(r"\bcontinue;", after), after[:200]
        assert re.search(r"__syncwarp\(\);\s*$", after), after[-200:]
    assert seen == 1


@pytest.mark.parametrize("name", ["prefix.cu", "tree.cu"])
def test_loops_of_unequal_length_before_what_the_whole_warp_does(name):
    # V's rows past the end are set to 0 by each lane as often as there is something for it
    code = _code(name)
    loops = list(re.finditer(r"for \(int idx = r; idx < [^;]*; idx \+= 128\)", code))
    assert len(loops) == 1
    for m in loops:
        _, end = _body(code, m.end())
        next_one = re.compile(WHOLE_WARP).search(code, end)
        assert "__syncwarp();" in code[end:next_one.start()]


@pytest.mark.parametrize("name", ["prefix.cu", "tree.cu"])
def test_the_other_slots_sums_are_read_between_fences(name):
    code = _code(name)
    votes = [m for m in re.finditer(r"ok = vote_all\(1, 256, ok\);", code) if "ex[r]" in code[m.end():m.end() + 200]]
    assert len(votes) == 1
    for m in votes:
        assert re.search(r"tc_fence_before\(\);\s*$", code[:m.start()])
        assert re.match(r"\s*if \(!ok\) (?:return false|break);\s*tc_fence_after\(\);", code[m.end():])
