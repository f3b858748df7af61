"""Every kernel that touches another CTA's shared memory first passes a cluster
barrier: only that shows that the other CTA has started.  Read from the sources,
since a missing barrier shows on a GPU by chance alone."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_rank_linear_02_b200", "csrc")
REMOTE = re.compile(r"\b(st_cluster_f32|ld_shared_cluster_v4|mbar_arrive_remote(_relaxed)?|bulk_signal_peer|"
                    r"tma_load_[23]d_pair|mma_commit_pair)\s*\(|(ld|st)\.shared::cluster\.[a-z0-9.]*f32")
BARRIER = re.compile(r"\b(cluster_sync_all|cluster_wait_started)\s*\(")


def kernels():
    """(file, name, body) of every __global__ function, comments taken out."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for g in re.finditer(r"__global__", text):
            start = text.index("{", g.end())
            depth, end = 1, start + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            name = re.findall(r"(\w+)\s*\((?!\()", text[g.end():start])
            name = next(n for n in name if n.endswith("kernel"))
            yield os.path.basename(path), name, text[start:end]


FOUND = list(kernels())
REMOTE_KERNELS = [(f, n, b) for f, n, b in FOUND if REMOTE.search(b)]


def test_the_cluster_kernels_are_found():
    names = {n for _, n, _ in REMOTE_KERNELS}
    assert {"distill_kernel", "epilogue_backward_kernel", "input_backward_kernel", "tc_small_kernel",
            "tc2_forward_kernel", "tc2t_forward_kernel"} <= names


@pytest.mark.parametrize("file,name,body", REMOTE_KERNELS, ids=[f"{f}:{n}" for f, n, _ in REMOTE_KERNELS])
def test_a_cluster_barrier_comes_before_the_first_remote_access(file, name, body):
    barrier = BARRIER.search(body)
    assert barrier is not None and barrier.start() < REMOTE.search(body).start(), f"{file}: {name}"
