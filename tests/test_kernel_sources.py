"""Rules that the CUDA sources keep by construction and that no run can show.
Read from the text; no GPU."""
import os
import re

import pytest

from mixture_experts_layer_56_b200 import build as B

# accesses to the shared memory of another CTA of the cluster
REMOTE = re.compile(r"\b(?:st_cluster_\w+|ld_cluster_\w+|ld_shared_cluster_\w+|mbar_arrive_cluster\w*)\s*\(")
BARRIER = re.compile(r"\b(?:cluster_sync_all|cluster_wait)\s*\(")


def kernels(path):
    """(line, body) of each __global__ function, comments removed."""
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"__global__", text):
        at, depth = text.index("{", m.end()), 0
        for end in range(at, len(text)):
            depth += (text[end] == "{") - (text[end] == "}")
            if depth == 0:
                break
        yield text.count("\n", 0, m.start()) + 1, text[at:end]


def test_the_kernels_are_found():
    assert sum(1 for p in B.sources() for _ in kernels(p)) >= 30


@pytest.mark.parametrize("path", B.sources(), ids=os.path.basename)
def test_no_remote_shared_memory_before_a_cluster_barrier(path):
    """A CTA's shared memory can be accessed from its cluster once it is known
    to have started, which the first cluster barrier shows."""
    for line, body in kernels(path):
        first = REMOTE.search(body)
        if first:
            barrier = BARRIER.search(body)
            assert barrier and barrier.start() < first.start(), (line, first.group())
