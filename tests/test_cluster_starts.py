"""The kernels' text, for what a run cannot show: an order that latencies alone hold up."""
import os
import re

import pytest

from bit_weight_streaming_q4_gb300 import build as qbuild


def kernels(name):
    """The bodies of a file's kernels, without comments."""
    with open(os.path.join(qbuild.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = {}
    for m in re.finditer(r"__global__[^{;]*?\b(\w+)\s*\(\s*const", text):
        at = text.index("{", m.end())
        depth, i = 1, at + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        found[m.group(1)] = text[at:i]
    return found


SHARING = sorted(f for f in os.listdir(qbuild.CSRC) if "map_shared_rank" in open(os.path.join(qbuild.CSRC, f)).read())


@pytest.mark.parametrize("name", SHARING)
def test_blocks_of_a_cluster_wait_for_one_another_before_they_share(name):
    """Another block's shared memory is there once that block has started: a barrier of the cluster comes first."""
    sharing = {k: b for k, b in kernels(name).items() if "map_shared_rank" in b}
    assert sharing
    for kernel, body in sharing.items():
        waits = re.search(r"\b\w+\.sync\(\)|barrier_wait\(|cluster_wait\(", body)
        assert waits and waits.start() < body.index("map_shared_rank"), kernel
