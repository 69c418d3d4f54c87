"""Loops with a barrier among some warps of a CTA, read from the kernels' sources.

Every wait on an mbarrier gives up after a limit; a named barrier (named_sync, named_and) has none.  So
the warps that meet at one inside a loop may not leave that loop on the outcome of a wait that each made for
itself: a warp that left would never arrive, and the others would stay.  They leave on what named_and
returns, which is the same for all of them.
"""
import glob
import os
import re

import pytest

from learnable_channel_permutation_b200 import build

SOURCES = sorted(glob.glob(os.path.join(build.CSRC, "*.cu")))


def _close(text, at, pair="{}"):
    """Index behind the bracket that closes the one at text[at]."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced brackets")


def _loops(text):
    """(header, body) of every for and while loop with a braced body."""
    for m in re.finditer(r"\b(?:for|while)\s*(?=\()", text):
        end = _close(text, m.end(), "()")
        brace = re.match(r"\s*\{", text[end:])
        if brace:
            start = end + brace.end() - 1
            yield text[m.end():end], text[start + 1:_close(text, start) - 1]


def _own(body):
    """The body without the loops inside it, whose breaks are their own."""
    for h, b in _loops(body):
        body = body.replace(h + " {" + b + "}", ";")
    return body


def _faults(text):
    """Exits of a loop with a named barrier that do not come from named_and."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    for header, body in _loops(text):
        own = _own(body)
        if not re.search(r"\bnamed_(sync|and)\(", own):
            continue
        waits = set(re.findall(r"\b(\w+) = [^;]*\bmbar_(?:try_)?wait", body))
        shared = set(re.findall(r"\b(\w+) = named_and\(", body))
        condition = header.split(";")[1] if header.count(";") == 2 else header
        yield from (f"loop condition on {w}" for w in waits - shared if re.search(rf"\b{w}\b", condition))
        for m in re.finditer(r"\bif \(([^;{}]*)\)\s*(?:\{\s*)?(?:break|return)\b", own):
            if "named_and(" not in m[1] and not any(re.search(rf"!{s}\b", m[1]) for s in shared):
                yield f"exit on ({m[1]})"


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(p) for p in SOURCES])
def test_warps_that_share_a_barrier_leave_its_loop_together(path):
    assert list(_faults(open(path).read())) == []


def test_the_reader_sees_lone_exits():
    lone = "for (int i = 0; i < n && ok; ++i) { named_sync(1, 128); ok = warp_all(mbar_wait(x, 0, f, 1)); }"
    jump = "for (;;) { named_sync(1, 128); for (int k = 0; k < n; ++k) { if (k) break; } ok = mbar_wait(x); if (!ok) break; }"
    fine = "for (int i = 0; i < n; ++i) { if (!named_and(1, 128, ok)) break; ok = mbar_wait(x); for (; k && ok;) { if (!ok) break; } }"
    also = "for (;;) { ok = named_and(1, 128, mbar_wait(x)); if (!ok) break; }"
    assert list(_faults(lone)) == ["loop condition on ok"] and list(_faults(jump)) == ["exit on (!ok)"]
    assert not list(_faults(fine)) and not list(_faults(also))
