"""What the kernels' sources have to keep to, where a run cannot show it."""
import os
import re

import pytest

from ternary_butterfly_experts_b200 import build


def kernels():
    """(name, body) of every __global__ function of the library."""
    for path in sorted(f for f in build.deps() if f.endswith((".cu", ".cuh"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__", text):
            at = text.index("{", text.index(")", re.compile(r"\w+_kernel\s*\(").search(text, m.end()).end()))
            depth, end = 0, at
            while True:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
                if depth == 0:
                    break
            yield os.path.basename(path) + ":" + re.search(r"(\w+_kernel)\s*\(", text[m.end():]).group(1), text[at:end]


REMOTE = re.compile(r'"(?:ld|st|red|atom)[\w.]*\.shared::cluster')
ARRIVE, WAIT = "barrier.cluster.arrive", "barrier.cluster.wait"
CASES = [(n, b) for n, b in kernels() if REMOTE.search(b)]


def test_cluster_kernels_are_found():
    assert {n.split(":")[1] for n, _ in CASES} == {"balance_finish_kernel", "bucket_cluster_kernel"}


@pytest.mark.parametrize("name,body", CASES, ids=[n for n, _ in CASES])
def test_blocks_of_a_cluster_have_started_before_their_memory_is_touched(name, body):
    """Another block's shared memory exists once that block runs, which a cluster barrier shows; and it goes when
    that block ends, so a barrier stands behind the last access too."""
    spots = [m.start() for m in REMOTE.finditer(body)]
    assert body.find(ARRIVE) >= 0 and body.find(ARRIVE) < body.find(WAIT) < spots[0]
    assert body.find(WAIT, body.find(ARRIVE, spots[-1])) > body.find(ARRIVE, spots[-1]) > spots[-1]
