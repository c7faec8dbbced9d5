"""A role that gives up waiting waits for its own products in flight before tensor memory is given back. A commit
covers what its own thread has issued, and products are issued by the lane that elect() names: the commit of the
drain has to be that lane's. (No wait is made to run out here: the sources are looked at. No GPU.)"""
import os
import re

import pytest

import matrix_dense_linear_spd_gb300 as bl

CSRC = os.path.join(os.path.dirname(bl.__file__), "csrc")


def blocks_around(text, at):
    """The heads of the blocks that hold text[at], the innermost first."""
    depth, heads = 0, []
    for i in range(at - 1, -1, -1):
        if text[i] == "}":
            depth += 1
        elif text[i] == "{":
            if depth:
                depth -= 1
            else:
                heads.append(text[max(text.rfind("\n", 0, i), text.rfind(";", 0, i)) + 1:i].strip())
    return heads


@pytest.mark.parametrize("name", ["xent_gemm.cuh", "orth_gemm.cuh"])
def test_the_issuing_lane_commits_the_drain(name):
    with open(os.path.join(CSRC, name)) as fh:
        text = re.sub(r"//[^\n]*", "", fh.read())
    commits = [m.start() for m in re.finditer(r"mma_commit_all<CTAS>\(&(\w+)", text)]
    products = [m.start() for m in re.finditer(r"tc::mma_f16<CTAS>\(", text)]
    assert len(commits) == 3 and products
    for at in commits + products:
        heads = blocks_around(text, at)
        assert any(h == "if (tc::elect())" for h in heads), heads[:3]
        assert not any("lane == 0" in h for h in heads), heads[:3]
