"""What the kernel before wrote is read by a dependent with loads that allow it, as the sources show."""
import os
import re

import pytest

from tests.test_launch_order_cpu import CSRC, bare


def body(text, name):
    """The function of this name, braces and all."""
    m = re.search(r"\b" + name + r"\s*\([^;{]*\)\s*\{", text)
    depth, i = 1, m.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[m.start():i]


@pytest.mark.parametrize("name", ["move_pages", "page_compact_kernel"])
def test_a_compaction_reads_its_plan_coherently(name):
    """The plan's kernel may still run when the moving one starts, so ld.global.nc (__ldg), which is for
    what nothing writes while a kernel lives, is not for the plan's sources and destinations."""
    text = body(bare(open(os.path.join(CSRC, "pages.cu")).read()), name)
    assert "pdl_wait()" in text or "p.src" in text
    assert "__ldg(" not in text
