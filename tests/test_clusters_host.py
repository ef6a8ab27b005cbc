"""Shared memory of another CTA of a cluster may be touched only when that CTA has begun: in
each kernel that does, a barrier of the whole cluster comes first. (Without one the result
depends on when CTAs are started, which no run shows; so this reads the sources.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_kv_selection_gb300", "csrc")
REMOTE = re.compile(r"map_shared_rank|\bat_rank<|\brank_shared<|\bpush_hist_row\(")
BARRIER = re.compile(r"\bcluster_begun\(\)|\bcluster\.sync\(\)|\bcluster_barrier<\w+>\(|\bhead_sync<\w+>\(|\bplanned\(\)")


def kernels():
    """Kernel names and their bodies, comments taken out."""
    for name in sorted(os.listdir(CSRC)):
        src = re.sub(r"//.*", "", open(os.path.join(CSRC, name)).read())
        for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", src):
            at = src.index("{", m.end())
            depth, end = 1, at + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(src[end], 0)
                end += 1
            yield m.group(1), src[at:end]


NAMES = ["attn_cluster_kernel", "cis_kernel", "find_kernel", "pages_kernel", "retrieve_kernel", "score_select_kernel"]


def test_every_such_kernel_is_named():
    assert sorted(n for n, body in kernels() if REMOTE.search(body)) == NAMES


@pytest.mark.parametrize("name", NAMES)
def test_a_barrier_before_another_ctas_memory(name):
    body = dict(kernels())[name]
    remote = REMOTE.search(body)
    assert remote, "reaches no other CTA"
    assert BARRIER.search(body, 0, remote.start()), body[:remote.end()][-300:]


def test_an_anchors_age_changes_once_all_ranks_have_read_it():
    """Ranks that read another age decide otherwise, and leave while the others still write to them."""
    body = dict(kernels())["cis_kernel"]
    assert body.index("= a.anchor_age !=") < body.index("a.anchor_age[qh] = ")
    calls = [m.start() for m in re.finditer(r"\brecord\(\d\)", body)]
    assert len(calls) == 3 and body.count("a.anchor_age[qh] = ") == 1
    for at in calls:                    # behind a barrier of the cluster, or where there is none
        before = body[:at].rstrip().splitlines()
        assert any("cluster.sync()" in x for x in before[-2:]) or before[-1].strip() == "if (!CLU)"
