"""Properties of the block operators' kernels that no run may bring out --
they would hang or fault a GPU, or depend on what another GPU maps -- read off
the sources instead."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_aware_optimizer_gb300", "csrc")
SOURCES = sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh", ".h")))


def _code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", SOURCES)
def test_no_load_is_multicast(name):
    """The library runs in replicas on several GPUs and takes any pointer a
    caller has, so no bulk or tensor load writes to several CTAs at once
    (arrivals on barriers may)."""
    joined = re.sub(r'"\s*"', "", _code(name))     # adjacent literals of one asm statement
    for statement in re.findall(r'"[^"]*cp\.async\.bulk[^"]*"', joined):
        assert "multicast" not in statement, statement


def _kernel(name, kernel):
    """The body of a __global__ function."""
    text = _code(name)
    start = text.index("{", text.index(kernel + "("))
    depth, end = 0, start
    while True:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
        if depth == 0:
            return text[start:end]


def test_cluster_sort_meets_before_it_writes_to_other_blocks():
    """A block's shared memory may be written by another block of its cluster
    only once it is known to have started."""
    body = _kernel("embedding.cu", "cluster_sort_kernel")
    first_store = re.search(r"\bst_cluster2?\(", body).start()
    met = re.search(r"\bcluster_(sync_all|wait)\(", body).start()
    assert met < first_store
    assert len(re.findall(r"\bcluster_arrive\w*\(", body)) == len(re.findall(r"\bcluster_wait\(", body))


def test_norm_gradient_leaves_no_thread_alone_at_a_barrier():
    """The warps of a row meet at barriers that have no time limit, so one
    whose bounded wait gave up says so in front of the step's reductions, and
    the whole row, which knows behind them, leaves at the next step's wait."""
    body = _kernel("block_norm_grad.cuh", "norm_backward_kernel")
    loop = body[body.index("int stage = 0;"):body.rindex("if (leave) return;")]
    for way in re.findall(r"[^;{}]*\b(?:break|return|goto \w+);", loop):
        assert way.strip() == "if (leave) break;", way
    asked, wait = loop.index("aborted = abort_flag"), loop.index("wait_bounded(")
    agreed, said = loop.index("row_failed[group] == before"), loop.index("row_failed[group] =", loop.index("if (leave)",
                                                                         loop.index("row_failed[group] == before")))
    assert asked < wait < agreed < said < loop.index("reduce(sums)")
    # the only other ways out: a row inside the warp, and the block's own agreement
    assert [" ".join(v.split()) for v in re.findall(r"leave = ([^;=][^;]*);", loop)] == [
        "false", "__syncthreads_or(abort_flag)", "(SIZE == 0 && tpr <= 32) || row_failed[group] == before"]
