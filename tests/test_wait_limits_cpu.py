"""Waits on barriers end after a time, as the sources show."""
import glob
import os
import re

import pytest

from tests.test_launch_order_cpu import CSRC, bare

TRY = re.compile(r"\b(?:mbar_try_wait|try_wait\w*|mbar_test_wait)\s*\(")


def closing(text, i):
    """Behind the bracket that closes the one at i."""
    pair = {"(": ")", "{": "}"}
    want, depth = text[i], 0
    while True:
        depth += {want: 1, pair[want]: -1}.get(text[i], 0)
        i += 1
        if depth == 0:
            return i


def statement(text, i):
    """Behind the statement that begins at i."""
    i += len(text[i:]) - len(text[i:].lstrip())
    if text[i] == "{":
        return closing(text, i)
    m = re.match(r"(?:for|while|if)\s*\(", text[i:])
    if m:
        return statement(text, closing(text, i + m.end() - 1))
    return text.index(";", i) + 1


def loops(text):
    """Loops that try a barrier, without what lies in loops inside of them that do."""
    found = [(m.start(), statement(text, m.start())) for m in re.finditer(r"\b(?:for|while)\s*\(", text)]
    for t in TRY.finditer(text):
        around = [x for x in found if x[0] < t.start() < x[1]]
        if around:
            a, b = max(around)
            yield text[a:b]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_a_loop_of_tries_looks_at_the_clock(path):
    """A try takes as long as the hardware likes, so that a number of them is no limit."""
    for loop in loops(bare(open(path).read())):
        assert "clock" in loop or "wait_slow(" in loop, loop


def test_the_sources_are_understood():
    found = {os.path.basename(p): len(list(loops(bare(open(p).read())))) for p in glob.glob(os.path.join(CSRC, "*.cu*"))}
    assert found["common.cuh"] and found["tc.cuh"] and found["kv8_attn_few.cu"]
