"""How a block of the gated scan's clusters leaves (CPU only).

Peers store into each other's shared memory, so a block may not end before every store into it has landed.
A block none of whose waits ran out has counted them all.  One that lost a wait has not; it gives them
time, and that pause has to stand behind the cluster's barrier: in front of it a late peer has yet to send
its last run.  The order cannot be seen in any result, so it is played through here, and read from the source.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_gated_delta_07_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, head):
    """The braces behind `head`."""
    at = text.index("{", text.index(head))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i]
    raise AssertionError(head)


def ending(text):
    """The order of the barrier and the pause at the block's end."""
    return [m for m in re.findall(r"cluster_sync|settle", body(text, "void leave("))]


def stays_long_enough(order, late_ms, way_ms=0.001, pause_ms=1.0):
    """Whether the lost block (at time 0) is still there when the last store of a peer, late by late_ms, lands."""
    now = 0.0
    for step in order:
        now = max(now, late_ms) if step == "cluster_sync" else now + pause_ms
    return now >= late_ms + way_ms


@pytest.mark.parametrize("late_ms", [0.0, 0.5, 1.0, 5.0, 1999.0])
def test_the_pause_covers_a_late_peer(late_ms):
    assert stays_long_enough(ending(source("gdr_scan.cuh")), late_ms)


def test_the_other_order_does_not():
    assert not stays_long_enough(["settle", "cluster_sync"], 5.0)


@pytest.mark.parametrize("name", ["gdr_scan_fwd.cu", "gdr_scan_bwd.cu"])
def test_the_kernels_leave_by_it(name):
    text = source(name)
    kernel = body(text, "scan_%s_kernel(" % name[9:12])
    assert kernel.rstrip().endswith("peers.leave(lost, CS, status);")
    assert kernel.count("cluster_sync") == 1 and "settle" not in kernel   # the one where every block has started
