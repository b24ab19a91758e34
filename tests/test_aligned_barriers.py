"""Aligned barriers in the kernels' sources.  A named or cluster barrier has to be executed by a
warp's lanes together; where one lane has run a long loop alone, only a __syncwarp() directly
before the instruction says so.  CPU only: the sources are read as text."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mxfp4_mixture_experts_softmax_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, name):
    """The text between the braces of the function `name`."""
    at = text.index("{", re.search(rf"\b{name}\([^)]*\)\s*{{", text).start())
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i]


@pytest.mark.parametrize("name,instruction", [("cluster_sync_all", "barrier.cluster.arrive"), ("all_at_barrier", "bar.red"),
                                              ("barrier_sync", "bar.sync"), ("barrier_arrive", "bar.arrive")])
def test_the_helpers_bring_the_warp_together(name, instruction):
    b = body(source("moe_device.cuh"), name)
    assert instruction in b
    assert "__syncwarp();" in b[:b.index(instruction)]


def test_cluster_barriers_come_from_the_helper():
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        if os.path.basename(path) != "moe_device.cuh":
            assert "barrier.cluster" not in source(os.path.basename(path)), path


@pytest.mark.parametrize("name", ["layer_few.cu", "linear_mxfp4.cu"])
def test_named_barriers_come_from_the_helpers(name):
    assert not re.search(r'"[^"]*\bbar\.(sync|arrive|red)', source(name))
