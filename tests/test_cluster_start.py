"""Clusters: a CTA's shared memory may be touched by the others only once it is
known to run.  Read from the sources, since a missing barrier shows no wrong
result as long as the CTAs happen to start together."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lm_head_linear_03_b200", "csrc")
REMOTE = ("st_cluster_", "mapa_shared(", "mbar_arrive_cluster(")


def kernels():
    """(name, body) of every kernel that reaches into another CTA's shared memory."""
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\s*\(", src):
            start = src.index("{", m.end())
            depth, end = 0, start
            while True:
                depth += {"{": 1, "}": -1}.get(src[end], 0)
                end += 1
                if depth == 0:
                    break
            body = src[start:end]
            if any(r in body for r in REMOTE):
                out.append((m.group(1), body))
    return out


def test_the_cluster_kernels_are_found():
    assert {k for k, _ in kernels()} == {"flce_pass1_kernel", "flce_pass2_kernel", "flce_logit_loss_kernel"}


@pytest.mark.parametrize("name,body", kernels(), ids=lambda x: x if x.endswith("_kernel") else "")
def test_a_cluster_barrier_comes_before_the_first_remote_access(name, body):
    first = min(body.index(r) for r in REMOTE if r in body)
    assert "cluster_sync_all()" in body[:first], name


def test_the_cluster_barrier_is_reached_by_whole_warps():
    src = open(os.path.join(CSRC, "sm100.cuh")).read()
    body = src[src.index("void cluster_sync_all()"):]
    assert body.index("__syncwarp()") < body.index("barrier.cluster.arrive")
