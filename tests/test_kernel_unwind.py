"""What a kernel does when one of its waits runs out, read from its source: no run reaches these paths (a wait has
seconds, its event microseconds), and none may be forced to."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_fa2_attn_gb300", "csrc")


def _code(name):
    """The file without comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def _enclosing(code, at):
    """Heads of the blocks around offset `at`, innermost first (what stands before each open brace)."""
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


def _landing_waits(code):
    """Offsets of the waits for copies to land, those a warp makes before it may leave its loops behind."""
    return [m.start() for m in re.finditer(r"mbar_wait\(&(?:bars->)?\w*full\w*(?:\[[^;]*?\])?, [^;]*tmo_unwind\)", code)]


def test_tree_producers_wait_for_their_copies_whatever_happens():
    # a role whose wait runs out after the producers' last issue would else let the CTA exit under copies in flight
    code = _code("tree.cu")
    waits = _landing_waits(code)
    assert len(waits) >= 3
    for at in waits:
        heads = _enclosing(code, at)
        assert not any("abort_flag" in h and h.startswith("if") for h in heads), heads[:3]


def test_tree_softmax_warps_keep_what_they_voted():
    # in a cluster the other CTAs join what is `finished`: all eight warps' partials, not those of the voter's own slot
    code = _code("tree.cu")
    votes = [m.start() for m in re.finditer(r"\bvote_all\(1, 256, ok\)", code)]
    assert len(votes) == 2
    for at in votes:
        assert re.search(r"[;{}]\s*ok = $", code[:at]), code[at - 40:at + 30]
    assert "bars->finished = ok;" in code


def test_every_producer_waits_for_its_copies_whatever_happens():
    for name, least in (("prefill_tc.cu", 3), ("decode.cu", 1), ("kv_outer.cu", 3), ("backward.cu", 8), ("tree.cu", 3)):
        code = _code(name)
        kept = [at for at in _landing_waits(code)
                if not any(re.fullmatch(r"if \((?:\*abort_flag|!ok)\)", h) for h in _enclosing(code, at))]
        assert len(kept) >= least and len(kept) == len(_landing_waits(code)), name
