"""Orders inside the kernels that a GPU run shows only by chance, read from the sources (CPU).

A CTA may write another CTA's shared memory once that CTA has started
(programming guide, distributed shared memory), and a cluster barrier is the
only thing that says so.
"""
import os
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


def _leaves(body):
    """Loops and roles that a warp leaves after a wait: (wait, text up to the break) outside single-thread blocks."""
    found, stack, start = [], [], 0
    for i, c in enumerate(body):
        if c == "{":
            stack.append(bool(re.search(r"elect_one\(\)|\bleader\b|\bthreadIdx\.x == 0|lane == 0", body[start:i])))
        elif c == "}":
            stack.pop()
        elif body.startswith("mbar_wait", i) and not any(stack):
            head = body[start:i + body[i:].index(";")]
            tail = body[i:]
            stop = re.search(r"\bbreak;|\n\s*__syncwarp\(\);", tail)
            if stop and tail[stop.start():].startswith("break"):
                found.append((head.strip(), head + tail[:stop.end()]))
        if c in "{};":
            start = i + 1
    return found


LEAVERS = {name: len(_leaves(body)) for name, body in S.kernels().items() if _leaves(body)}


def test_the_kernels_that_leave_waits_are_found():
    assert LEAVERS == {"gemm_block_tile_kernel": 2, "gemm_block_decode_kernel": 5, "moe_up_kernel": 3, "moe_down_kernel": 3,
                       "gemm_tile_kernel": 1, "gemm_pair_kernel": 1, "w4a16_kernel": 2}


@pytest.mark.parametrize("name", sorted(LEAVERS))
def test_a_warp_leaves_a_wait_as_one(name):
    # a limit that runs out between two lanes' polls must not split a warp before tcgen05.ld or __syncwarp
    for wait, until_break in _leaves(S.kernels()[name]):
        assert "__all_sync(" in until_break, wait


@pytest.mark.parametrize("name", ["gemm_block_decode_kernel", "moe_up_kernel", "moe_down_kernel"])
def test_column_scales_are_ordered_before_their_readers(name):
    # a lane writes its columns of cs, promote reads all of them in every lane: a vote or a barrier's
    # poll between them orders no shared memory
    body = S.kernels()[name]
    writes = [m.end() for m in re.finditer(r"\bcs\[[^]]*\] = ", body)]
    assert writes
    for at in writes:
        use = re.search(r"\bpromote\(", body[at:])
        assert "__syncwarp();" in body[at:at + use.start()]


def test_the_tile_kernels_promotion_votes_behind_a_tile():
    # it stays in the group loop with what each lane knows, hands no buffer back after a failed wait,
    # and leaves by a vote
    promotion = S.roles(S.kernels()["gemm_block_tile_kernel"])[-1]
    wait = promotion.index("ok = ok && mbar_wait_short(")
    arrive = promotion.index("mbar_arrive_relaxed(&tempty_bar[buf])")
    leave = promotion.index("if (!__all_sync(0xffffffffu, ok)) break;")
    assert wait < arrive < leave < promotion.index("tma_store_2d")
    assert "if (lane == 0 && ok)" in promotion[wait:arrive] and "break;" not in promotion[wait:leave]
    assert promotion.count("mbar_wait") == 1


def test_only_weight_scales_are_read_as_constant_data():
    # with programmatic launch an earlier kernel may write activations, their scales, biases and outputs
    # while a kernel is resident, so only the weights' side may go through the read-only path
    # (the smoothing multipliers of q8_quant.cu are no kernel's output)
    files = sorted(os.listdir(S.CSRC))
    assert len(files) > 10
    for f in files:
        s = S.text(f)
        assert s.count("__ldg(") == (2 if f == "q8_quant.cu" else 0)
        for m in re.finditer(r"\.nc\b", s):
            assert re.findall(r"float (\w+)\(", s[:m.start()])[-1] == "ld_weight_scale"
        for arg in re.findall(r"[^t] ld_weight_scale\(([^;]*)\);", s):
            assert arg.startswith("sw")


def test_streamed_inputs_are_not_loaded_before_the_wait():
    # a load that is not volatile may be moved over the wait for the kernel that writes the input
    for f in sorted(os.listdir(S.CSRC)):
        for m in re.finditer(r"asm(\s+volatile)?\s*\(\s*\"ld\.global", S.text(f)):
            assert m.group(1), f
