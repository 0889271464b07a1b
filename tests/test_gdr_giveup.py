"""What the gated delta rule's kernels leave behind when a bounded wait gives up.

A role that issued copies or products has to see them complete before the CTA
exits, on the path that gave up too: a load still on its way would land in the
shared memory of the CTA that comes next, a product in TMEM that is no longer
this one's.  The path takes a wait of 2 s, with copies in flight longer than
any copy takes, so it is checked here by reading the kernels' sources: each of
these roles ends with an unconditional drain().  (tests/test_gdr_gpu.py and
tests/test_gdr_paths_gpu.py run the waits out with nothing left in flight.)
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_momentum_b200", "csrc")


def _branch(src, head):
    """The text of the block that `head` opens."""
    i = src.index(head) + len(head)
    depth, j = 1, i
    while depth:
        depth += {"{": 1, "}": -1}.get(src[j], 0)
        j += 1
    return src[i:j - 1]


def _ends_with_drain(block):
    """The block's last statement is a drain that no earlier wait's outcome guards."""
    block = re.sub(r"//[^\n]*", "", block).rstrip()
    while block.endswith("}"):                      # the blocks that end here: `if (lane == 0) { ... }` or a plain scope
        block = block[:-1].rstrip()
    last = block[block.rindex(";", 0, len(block) - 1) + 1:]
    return "drain(" in last and "live" not in last and "abort" not in last


ROLES = [("gdr_chain.cu", "if (warp == W_PROD) {"), ("gdr_chain.cu", "else if (warp == W_MMA) {"),
         ("gdr_bwd.cu", "if (w == G_LOAD) {"), ("gdr_bwd.cu", "else if (w == G_MMA) {")]


@pytest.mark.parametrize("name, head", ROLES, ids=lambda x: x.split("==")[-1].strip(" ){") if "==" in x else x)
def test_roles_wait_for_what_they_issued(name, head):
    with open(os.path.join(CSRC, name)) as f:
        src = f.read()
    block = _branch(src, head)
    assert _ends_with_drain(block), f"{name}: {head} leaves without waiting"


def test_preparing_kernel_waits_for_its_copies():
    with open(os.path.join(CSRC, "gdr_fwd.cu")) as f:
        src = f.read()
    block = _branch(src, "if (!__syncthreads_and(mbar_wait_sleep(bar, 0, &g_prep_dev_err))) {")
    assert "drain(bar, 0" in block and block.index("drain(") < block.index("return")
