"""What the prefix kernel does when one of its waits runs out, read from its source: no run reaches these paths (a wait
has seconds, its event microseconds), and none may be forced to."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_fa2_attn_gb300", "csrc")


def _code():
    """The file without comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "prefix.cu")).read())


def _blocks(code, at):
    """Heads of the blocks around offset `at`, innermost first."""
    heads, depth = [], 0
    for i in range(at, -1, -1):
        if code[i] == "}":
            depth += 1
        elif code[i] == "{":
            if depth:
                depth -= 1
            else:
                heads.append(re.split(r"[;{}]", code[:i])[-1].strip())
    return heads


def test_copies_land_before_the_block_leaves():
    # whether or not a wait has run out so far: another role's may after the last copy was issued
    code = _code()
    waits = [m.start() for m in re.finditer(r"mbar_wait_lean\(&\w+(?:->\w+)?(?:\[[^;]*?\])?, [^;]*tmo_unwind\)", code)]
    assert len(waits) == 3  # Q, the K or V ring, the last MMAs
    for at in waits:
        assert not any("abort_flag" in h or "ok" in h for h in _blocks(code, at)), _blocks(code, at)[:3]


def test_softmax_warps_keep_what_they_voted():
    code = _code()
    votes = [m.start() for m in re.finditer(r"\bvote_all\(1, 256, ok\)", code)]
    assert len(votes) == 3  # before a segment, at the end of a narrow and of a slim one
    for at in votes:
        assert re.search(r"[;{}]\s*ok = $", code[:at]), code[at - 40:at + 30]


def test_lanes_of_a_warp_leave_together():
    # a lane that leaves its loop alone would keep the others in their next warp-wide instruction for good
    code = _code()
    for m in re.finditer(r"mbar_(?:wait_lean|test)\(", code):
        line = code[code.rindex("\n", 0, m.start()) + 1:code.index("\n", m.start())]
        if "tmo_unwind" in line or "__all_sync(0xffffffffu," in line:
            continue
        # the walk is one lane's; the MMA issuer's lanes meet at the head of its loop over segments
        assert "seg_empty" in line or re.match(r"\s*auto wwait = .* return mbar_wait_lean\(bar, parity, tmo, abort_flag\); };$", line), line
    assert "for (int nt; __all_sync(0xffffffffu, ok); g += nt)" in code
    assert "while (__all_sync(0xffffffffu, ok && !*abort_flag))" in code
