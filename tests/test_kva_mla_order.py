"""Order of the accesses to the array that the softmax warps of the MLA kernel
share, read off the source.

Each of the four warps writes the factors of its own heads and reads those of
all heads.  What a warp reads has to be behind a vote of the four after it was
written, and what it overwrites behind one that every reader has reached: a
vote, or its own arrival on p_full followed by a wait for pv_done, which
completes only when all four have arrived."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "gqa_kv_cache_mla_gb300", "csrc", "mla_decode_paged.cu")

EVENTS = [("write", r"sm\.alpha\[[^\]]*\] = "), ("read", r"= sm\.alpha\["),
          ("vote", r"any_softmax\("), ("arrive", r"mbar_arrive\(&sm\.p_full\)"),
          ("wait", r"wait_phase\(&sm\.pv_done")]


def events(text):
    at = []
    for name, pattern in EVENTS:
        at += [(m.start(), name) for m in re.finditer(pattern, text)]
    return [name for _, name in sorted(at)]


def first_fault(names):
    """Index of the first access that is not ordered behind the others', or None."""
    unread = unwritten = False  # a read no overwrite may pass, a write no read may pass
    arrived = False
    for i, name in enumerate(names):
        if name == "vote":
            unread = unwritten = arrived = False
        elif name == "arrive":
            arrived = True
        elif name == "wait":
            unread = unread and not arrived
        elif name == "write":
            if unread:
                return i
            unwritten = True
        else:
            if unwritten:
                return i
            unread, arrived = True, False
    return None


def test_rule():
    assert first_fault(["write", "vote", "read", "arrive", "wait", "write", "vote", "read"]) is None
    assert first_fault(["write", "vote", "read", "arrive", "write"]) == 4
    assert first_fault(["write", "vote", "read", "wait", "write"]) == 4
    assert first_fault(["write", "read"]) == 1


def test_factors_of_the_softmax_warps():
    text = open(SOURCE).read()
    body = text[text.index("void soften("):]
    body = re.sub(r"//[^\n]*", "", body[:body.index("\ntemplate")])
    names = events(body)
    assert names.count("write") == 4 and names.count("read") == 2
    assert first_fault(names + names) is None  # and on to the next segment
