"""Programmatic dependents wait before they can leave, as their sources show."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "draft_block_candidate_gb300", "csrc")


def bare(text):
    """Without comments."""
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def kernels():
    """{name: text from its parameters to the next kernel or the end of its file}"""
    out = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        for piece in bare(open(path).read()).split("__global__")[1:]:
            m = re.search(r"(\w+)\s*\((?!\s*\w*\s*\))(?=[^;{]*\)\s*\{)", re.sub(r"__launch_bounds__\([^{]*?\)\s*(?=\w+\()", "", piece))
            out[m.group(1)] = piece
    return out


def dependents():
    """Kernels that launch_k may launch before the one ahead of them has ended."""
    names = set()
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        text = bare(open(path).read())
        for m in re.finditer(r"launch_k\(\s*(\w+)", text):
            name = m.group(1)
            if name in ("k", "kern", "KERNEL"):  # chosen before: the unit's kernels that are launched in no other way
                plain = set(re.findall(r"(\w+_kernel)\s*(?:<[^<>;]*>)?\s*<<<", text))
                names |= {n for n in re.findall(r"(\w+_kernel)\s*<", text)} - plain
            else:
                names.add(name)
    return names & set(kernels())


def test_the_sources_are_understood():
    assert {"kv8_join_kernel", "beam_merge_kernel", "logit_pass_kernel", "gemm_tc_kernel", "greedy_walk_kernel"} <= dependents()


@pytest.mark.parametrize("name", sorted(dependents()))
def test_a_dependent_waits_before_it_can_leave(name):
    """A dependent's end is taken for its predecessor's too, so no thread may return ahead of the wait."""
    ahead, wait, _ = kernels()[name].partition("pdl_wait()")
    assert wait, "no wait"
    assert not re.search(r"\breturn\b", ahead)
