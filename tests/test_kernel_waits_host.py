"""Waits of the kernels that end, read from their sources (no GPU).

A wait on a memory barrier gives up after a limit, and its warp then leaves its loop.  A barrier
of several warps inside such a loop has no limit: the warps have to leave together, by a vote
(epi_any), or the ones that go on wait for one that has left.
"""
import glob
import os
import re

import pytest

from addmm_implicit_im2col_gb300 import build

SOURCES = sorted(glob.glob(os.path.join(build.CSRC, "*.cu")))


def code(path):
    with open(path) as f:
        text = f.read()
    return re.sub(r"//[^\n]*", "", text)


def kernels(text):
    """The text of each __global__ function, up to the next one, by name."""
    parts = re.split(r"(?=__global__\s)", text)[1:]
    return {re.search(r"\b(k_\w+)\s*\(", p).group(1): p for p in parts}


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_barriers_of_a_role_come_with_a_vote(path):
    for name, body in kernels(code(path)).items():
        if re.search(r"\bepi_sync\s*\(", body):
            assert re.search(r"if\s*\((tc::)?epi_any\s*\(", body), f"{name}: epi_sync without a vote on leaving"


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_named_barriers_are_the_common_ones(path):
    assert not re.search(r"\bbar\.(sync|red|arrive)\b", code(path))


def test_roles_of_the_adapters_wait_for_the_launch_before_by_themselves():
    """The weights' gradients may run for seconds where one adapter has all of many rows: the second
    product, which starts beside their end, may not count that against its own waits' limit."""
    body = kernels(code(os.path.join(build.CSRC, "k_adapters.cu")))["k_adapters_up"]
    roles = re.split(r"\}\s*else if \(warp == UP_EPI \+ LOAD\) \{|\}\s*else \{\s*const int q4", body)
    assert len(roles) == 3
    for role in roles:
        # what another role makes of the launch before: h, w and the accumulators
        limited = [m.start() for m in re.finditer(r"warp_wait_bar\(&ctl\.(accf|acce|hfull|hempty|wfull|wempty)", role)]
        assert limited and 0 <= role.find("griddep_wait()") < limited[0]
