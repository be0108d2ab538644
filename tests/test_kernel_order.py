"""Orders inside the kernels that a GPU run shows only by chance, read from the sources (CPU).

A CTA may write another CTA's shared memory once that CTA has started
(programming guide, distributed shared memory), and a cluster barrier is the
only thing that says so.
"""
import re

import pytest

from tests import kernel_source as S

REMOTE = re.compile(r"\b(st_shared_cluster_\w+|mbar_arrive_cluster)\s*\(")
WRITERS = ["gemm_block_decode_kernel", "gemm_decode_kernel", "gemm_pair_kernel", "w4a16_kernel"]


def test_every_kernel_that_writes_remotely_is_listed():
    assert sorted(k for k, body in S.kernels().items() if REMOTE.search(body)) == sorted(WRITERS)


@pytest.mark.parametrize("name", WRITERS)
def test_remote_shared_memory_after_the_cluster_started(name):
    body = S.kernels()[name]
    first = REMOTE.search(body)
    assert first, "writes no other CTA's shared memory: not for this list"
    before = body[:body.index("if (warp == 0) {")]
    if "cluster_sync()" in before:          # one barrier of all threads, before the roles part
        return
    assert before.count("cluster_started()") == 1
    for role in S.roles(body):              # a thread that arrived waits once, before what it writes
        assert role.count("cluster_wait_started()") == 1
        write = REMOTE.search(role)
        assert write is None or role.index("cluster_wait_started()") < write.start()
